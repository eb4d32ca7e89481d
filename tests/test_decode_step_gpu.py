"""One decoder layer's step as a serving program runs it on 4-bit storage:
fused projection with adapters, append to the cache, attention, output
projection with adapters, mixture of experts; each step checked against its
definition on the inputs it was given, and the whole run captured and replayed."""
import numpy as np
import pytest
import torch

from post_weight_quantization_11_b200 import gptq as G
from tests import decode_ref as R
from tests.test_kv4_gpu import _attn_ref, _np, _table

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _t(a):
    if a is None:
        return None
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int32) if a.dtype == np.uint32 else a).to(DEV)


class Layer:
    """Weights, cache and buffers of one layer for B sequences of n tokens each"""

    def __init__(self, rng, B, n, d=512, hq=8, hkv=2, D=64, f=384, E=4, r=8, page=16, width=6):
        self.B, self.n, self.d, self.hq, self.hkv, self.D = B, n, d, hq, hkv, D
        T = B * n
        self.host = dict(qkv=R.packed_layer(rng, (hq + 2 * hkv) * D, d, 128, True),
                         out=R.packed_layer(rng, d, hq * D, 64),
                         inn=R.packed_layer(rng, 2 * f, d, 128, lead=(E,)),
                         down=R.packed_layer(rng, d, f, 128, lead=(E,)))
        self.lay = {k: {x: _t(v[x]) for x in ("qw", "sc", "qz", "perm")}
                    for k, v in self.host.items()}
        ab = lambda o, i: ((rng.standard_normal((3, r, i)) * 0.02).astype(np.float16),   # noqa
                           (rng.standard_normal((3, o, r)) * 0.02).astype(np.float16))
        self.qkv_ab, self.out_ab = ab((hq + 2 * hkv) * D, d), ab(d, hq * D)
        self.scaling = np.array([1.0, 2.0, 0.5], np.float32)
        self.ids = np.repeat(rng.integers(-1, 3, B), n).astype(np.int32)
        self.order = rng.permutation(B * width).reshape(B, width).astype(np.int32)
        self.page = page
        self.cache = G.KV4Cache.empty(B * width, hkv, page, D, 32, DEV)
        self.table = _table(page * width, D)
        self.x = torch.zeros(T, d, dtype=torch.float16, device=DEV)
        self.pos = torch.zeros(T, dtype=torch.int32, device=DEV)
        self.slots = torch.zeros(T, dtype=torch.int64, device=DEV)
        self.lens = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.start = _t(np.arange(0, T + 1, n, dtype=np.int32))
        self.logits = torch.zeros(T, E, device=DEV)
        self.dev = [_t(v) for v in (*self.qkv_ab, *self.out_ab, self.scaling, self.ids, self.table,
                                    self.order)]

    def inputs(self, rng, before):
        T = self.B * self.n
        x = rng.standard_normal((T, self.d)).astype(np.float16)
        pos = np.concatenate([np.arange(p, p + self.n) for p in before]).astype(np.int32)
        seq = np.repeat(np.arange(self.B), self.n)
        slots = self.order[seq, pos // self.page].astype(np.int64) * self.page + pos % self.page
        lg = rng.standard_normal(self.logits.shape).astype(np.float32)
        for dst, src in ((self.x, x), (self.pos, pos), (self.slots, slots), (self.logits, lg),
                         (self.lens, np.asarray(before, np.int32) + self.n)):
            dst.copy_(torch.from_numpy(src))
        return x, pos, slots, lg

    def step(self):
        a1, b1, a2, b2, sc, ids, table, order = self.dev
        hq, hkv, D = self.hq, self.hkv, self.D
        L = self.lay
        qkv = G.gptq_w4a16_lora(self.x, L["qkv"]["qw"], L["qkv"]["sc"], L["qkv"]["qz"], a1, b1, ids,
                                sc, 128, L["qkv"]["perm"]).view(-1, hq + 2 * hkv, D)
        q, _, _ = G.gptq_kv4_append(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], self.pos, self.slots,
                                    table, self.cache, q=qkv[:, :hq])
        o = G.gptq_kv4_attention(q, self.cache, order, self.lens, self.start, D ** -0.5,
                                 max_q_len=self.n)
        y = G.gptq_w4a16_lora(o.view(-1, hq * D), L["out"]["qw"], L["out"]["sc"], L["out"]["qz"], a2,
                              b2, ids, sc, 64)
        h = (self.x.float() + y * 0.05).half()
        z = G.gptq_w4a16_moe(h, self.logits, L["inn"]["qw"], L["inn"]["sc"], L["inn"]["qz"],
                             L["down"]["qw"], L["down"]["sc"], L["down"]["qz"], 2, 128)
        return qkv, q, o, y, h, z


def _check(lay, got, x, pos, slots, lg):
    qkv, q, o, y, h, z = (t.cpu().numpy() for t in got)
    T, D, hq = len(x), lay.D, lay.hq
    ref, bound = R.lora(x, lay.host["qkv"], *lay.qkv_ab, lay.scaling, lay.ids)
    assert (np.abs(qkv.reshape(T, -1) - ref) <= bound).all()
    assert np.array_equal(q, R.rotate(qkv[:, :hq], pos, lay.table, False, np.float32).astype(np.float16))
    c = dict(q=q, cache=lay.cache, raw=_np(lay.cache), table=lay.order, page=lay.page, D=D,
             lens=list(lay.lens.cpu().numpy()), start=list(lay.start.cpu().numpy()), scale=D ** -0.5)
    ref, bound = _attn_ref(c)
    assert (np.abs(o - ref) <= bound).all()
    ref, bound = R.lora(o.reshape(T, -1), lay.host["out"], *lay.out_ab, lay.scaling, lay.ids)
    assert (np.abs(y - ref) <= bound).all()
    ref, bound = R.moe(h, lg, 2, True, lay.host["inn"], lay.host["down"])
    assert (np.abs(z - ref) <= bound).all()


@pytest.mark.parametrize("B,n", [(1, 1), (5, 1), (3, 4), (2, 20)])
def test_steps_of_a_layer(B, n):
    rng = np.random.default_rng(B * 10 + n)
    lay = Layer(rng, B, n)
    before = np.zeros(B, int)
    for _ in range(3):                                        # a prompt, then more tokens
        inp = lay.inputs(rng, before)
        _check(lay, lay.step(), *inp)
        before = before + n


def test_captured_step_replays_as_the_sequences_grow():
    rng = np.random.default_rng(99)
    lay = Layer(rng, 4, 1)
    lay.inputs(rng, [0] * 4)
    lay.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = lay.step()
    for t in range(1, 20):
        inp = lay.inputs(rng, [t] * 4)
        graph.replay()
        if t in (1, 15, 16, 19):
            torch.cuda.synchronize()
            _check(lay, got, *inp)


def test_two_streams_at_once():
    """The same layer's calls on two streams, each with its own buffers."""
    rng = np.random.default_rng(100)
    lays = [Layer(rng, 3, 1) for _ in range(2)]
    inp = [lay.inputs(rng, [0, 0, 0]) for lay in lays]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for lay, st in zip(lays, streams):
        with torch.cuda.stream(st):
            got.append(lay.step())
    torch.cuda.synchronize()
    for lay, g, i in zip(lays, got, inp):
        _check(lay, g, *i)


def test_calls_back_to_back_equal_calls_one_by_one():
    """Kernels begin while the ones before them end: a chain of calls, each on the last
    one's output and all in one workspace, gives what it gives with a wait in between
    (eagerly, in two streams at once and replayed)."""
    rng = np.random.default_rng(41)
    d, f, E = 1024, 512, 8
    lay, inn, down = (R.packed_layer(rng, *s) for s in ((d, d, 64, True), (2 * f, d, 64, True, False, (E,)),
                                                        (d, f, 64, False, False, (E,))))
    dv = {n: [_t(v[k]) for k in ("qw", "sc", "qz", "perm")]
          for n, v in (("lay", lay), ("inn", inn), ("down", down))}
    a = _t((rng.standard_normal((5, 32, d)) * 0.02).astype(np.float16))
    b = _t((rng.standard_normal((5, d, 32)) * 0.02).astype(np.float16))
    scaling = _t(np.array([1.0, -2.0, 0.5, 1.5, 0.25], np.float32))
    x = _t(rng.standard_normal((60, d)).astype(np.float16))
    ids = _t(rng.integers(-1, 5, 60).astype(np.int32))
    logits = _t(rng.standard_normal((60, E)).astype(np.float32))
    logits[3] = float("-inf")                               # a token without experts
    nbytes = max(G.gptq_w4a16_lora_workspace_bytes(T, d, d, 64, 32) for T in (1, 7, 16, 17, 33, 60))
    nbytes = max(nbytes, G.gptq_w4a16_moe_workspace_bytes(60, E, 2, d, f))

    def chain(ws, wait):
        h, all_y = x, []
        for T in (60, 7, 33, 1, 17, 60, 16):
            q, s, z, perm = dv["lay"]
            y = G.gptq_w4a16_lora(h[:T], q, s, z, a, b, ids[:T], scaling, 64, perm if T != 7 else None, ws=ws)
            wait()
            m = G.gptq_w4a16_moe(torch.tanh(y).half(), logits[:T], *dv["inn"][:3], *dv["down"][:3], 2, 64,
                                 perm_in=dv["inn"][3], ws=ws)
            wait()
            all_y += [y, m]
            h = torch.cat([torch.tanh(m).half(), x[T:]])
        return all_y

    space = [torch.full((nbytes,), 255, dtype=torch.uint8, device=DEV) for _ in range(2)]
    want = chain(space[0], torch.cuda.synchronize)
    none = lambda: None                                    # noqa: E731
    for _ in range(3):
        assert all(torch.equal(u, v) for u, v in zip(chain(space[0], none), want))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for st, ws in zip(streams, space):
        with torch.cuda.stream(st):
            got.append([chain(ws, none) for _ in range(2)])
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for runs in got for run in runs for u, v in zip(run, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(space[0], none)
    for k in range(2):
        space[0].fill_(255 * k)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(out, want))
