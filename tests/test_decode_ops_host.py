"""Host-side checks of the decode-step entry points (no GPU): bad arguments are
refused before anything is launched, calls with nothing to do return at once,
and the workspace sizes are monotone and never zero for real calls."""
import ctypes

import pytest

from post_weight_quantization_11_b200 import gptq as G

FAKE = ctypes.c_void_p(1 << 20)          # 16-byte aligned, never dereferenced
MIS = ctypes.c_void_p((1 << 20) + 4)
ODD = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    import torch
    if torch.cuda.is_available():
        pytest.skip("host-side argument checks with fake pointers run where no GPU is visible")
    from post_weight_quantization_11_b200 import build
    build.build()
    return G.load_library()


def _caller(fn, names, defaults):
    def call(**kw):
        a = dict(defaults)
        assert set(kw) <= set(names), set(kw) - set(names)
        a.update(kw)
        return fn(*[a[n] for n in names])
    return call


def test_lora(lib):
    ws = G.gptq_w4a16_lora_workspace_bytes(4, 64, 256, 128, 8)
    assert ws > 0 and G.gptq_w4a16_lora_workspace_bytes(0, 64, 256, 128, 8) == 0
    assert G.gptq_w4a16_lora_workspace_bytes(400, 64, 256, 128, 8) > ws
    names = ("x batch qw sc qz perm m d g a b scaling adapter n rank y ws wsb stream").split()
    c = _caller(lib.gptq_w4a16_lora, names,
                dict(x=FAKE, batch=4, qw=FAKE, sc=FAKE, qz=FAKE, perm=None, m=64, d=256, g=128,
                     a=FAKE, b=FAKE, scaling=FAKE, adapter=FAKE, n=2, rank=8, y=FAKE, ws=FAKE,
                     wsb=ws, stream=None))
    for p in ("x", "qw", "sc", "qz", "y", "ws", "a", "b", "scaling", "adapter"):
        assert c(**{p: None}) == 1
    for p in ("x", "qw", "sc", "qz", "y", "ws", "a", "b", "perm"):
        assert c(**{p: MIS}) == 1
    assert c(adapter=ODD) == 1 and c(scaling=ODD) == 1
    assert c(wsb=ws - 1) == 1
    for bad in (dict(batch=-1), dict(batch=65536), dict(d=200), dict(d=64), dict(d=32896), dict(m=0),
                dict(n=-1), dict(n=65537), dict(m=(1 << 24) + 1)):
        assert c(**bad) == 2
    for bad in (dict(g=48), dict(g=16), dict(g=0), dict(g=512), dict(g=96), dict(rank=4),
                dict(rank=0), dict(rank=12), dict(rank=264)):
        assert c(**bad) == 4
    assert c(batch=0, x=None, y=None, adapter=None) == 0
    assert c(batch=0, d=200) == 2                             # still a bad layer


def test_moe(lib):
    ws = G.gptq_w4a16_moe_workspace_bytes(4, 8, 2, 256, 384)
    assert ws >= 4 * 2 * 384 * 4 and G.gptq_w4a16_moe_workspace_bytes(0, 8, 2, 256, 384) == 0
    names = ("x T logits E k renorm qi si zi pi qo so zo po d f g y ws wsb stream").split()
    c = _caller(lib.gptq_w4a16_moe, names,
                dict(x=FAKE, T=4, logits=FAKE, E=8, k=2, renorm=1, qi=FAKE, si=FAKE, zi=FAKE, pi=None,
                     qo=FAKE, so=FAKE, zo=FAKE, po=None, d=256, f=384, g=128, y=FAKE, ws=FAKE, wsb=ws,
                     stream=None))
    for p in ("x", "logits", "qi", "si", "zi", "qo", "so", "zo", "y", "ws"):
        assert c(**{p: None}) == 1
    for p in ("x", "qi", "si", "zi", "qo", "so", "zo", "y", "ws", "pi", "po"):
        assert c(**{p: MIS}) == 1
    assert c(logits=ODD) == 1 and c(wsb=ws - 1) == 1
    for bad in (dict(T=-1), dict(E=0), dict(k=0), dict(d=200), dict(f=200), dict(f=0), dict(d=32896)):
        assert c(**bad) == 2
    for bad in (dict(T=65), dict(E=257), dict(k=9, E=16), dict(k=3, E=2), dict(g=48), dict(g=256),
                dict(g=-2)):
        assert c(**bad) == 4
    assert c(T=0, x=None, logits=None, y=None) == 0


def test_append(lib):
    names = ("q qs k ks v vs dt T hq hkv D pos slots table npos rot inter g pages page kc kp vc vp qo "
             "kval vval stream").split()
    c = _caller(lib.gptq_kv4_append, names,
                dict(q=FAKE, qs=512, k=FAKE, ks=512, v=FAKE, vs=512, dt=1, T=4, hq=4, hkv=2, D=64,
                     pos=FAKE, slots=FAKE, table=FAKE, npos=100, rot=64, inter=0, g=32, pages=4, page=16,
                     kc=FAKE, kp=FAKE, vc=FAKE, vp=FAKE, qo=FAKE, kval=None, vval=None, stream=None))
    for p in ("k", "v", "slots", "table", "pos", "kc", "kp", "vc", "vp", "qo", "q"):
        assert c(**{p: None}) == 1
    for p in ("q", "k", "v", "table", "kc", "kp", "vc", "vp", "qo"):
        assert c(**{p: MIS}) == 1
    assert c(slots=MIS) == 1 and c(pos=ODD) == 1
    assert c(kval=FAKE) == 1 and c(vval=FAKE) == 1            # both or neither
    assert c(dt=2) == 1
    for p in ("qs", "ks", "vs"):
        assert c(**{p: 64}) == 1                              # shorter than a token's rows
        assert c(**{p: 516}) == 1                             # not a multiple of 16 bytes
    for bad in (dict(T=-1), dict(hkv=0), dict(hq=0), dict(hq=1025), dict(pages=0), dict(npos=0)):
        assert c(**bad) == 2
    for bad in (dict(D=96), dict(D=32), dict(g=16), dict(g=128), dict(g=48), dict(rot=8), dict(rot=80),
                dict(rot=-16), dict(page=24), dict(page=8), dict(page=8192)):
        assert c(**bad) == 4
    assert c(T=0, q=None, qo=None, k=None, v=None, slots=None, pos=None) == 0


def test_attention(lib):
    W = G.gptq_kv4_attention_workspace_bytes
    ws = W(2, 8, 2, 64, 1, 64000)
    assert ws > 0 and W(0, 8, 2, 64, 1, 64000) == 0
    assert W(2, 8, 2, 64, 1, 64) == 0                         # one chunk: nothing to join
    names = ("q T B hq hkv D kc kp vc vp pages page g table width lens start scale window maxq maxl out ws "
             "wsb stream").split()
    c = _caller(lib.gptq_kv4_attention, names,
                dict(q=FAKE, T=2, B=2, hq=8, hkv=2, D=64, kc=FAKE, kp=FAKE, vc=FAKE, vp=FAKE, pages=9,
                     page=16, g=32, table=FAKE, width=4, lens=FAKE, start=FAKE, scale=0.125, window=0,
                     maxq=1, maxl=64, out=FAKE, ws=FAKE, wsb=ws, stream=None))
    for p in ("q", "kc", "kp", "vc", "vp", "table", "lens", "start", "out"):
        assert c(**{p: None}) == 1
    long = dict(maxl=64000, width=4000)
    assert c(ws=None, **long) == 1 and c(wsb=ws - 1, **long) == 1
    for p in ("q", "kc", "kp", "vc", "vp", "out", "ws"):
        assert c(**{p: MIS}) == 1
    for p in ("table", "lens", "start"):
        assert c(**{p: ODD}) == 1
    assert c(scale=float("nan")) == 1 and c(scale=float("inf")) == 1
    for bad in (dict(T=-1), dict(B=-1), dict(B=65536), dict(hq=7), dict(hq=0), dict(hkv=0), dict(pages=0),
                dict(width=-1), dict(window=-1), dict(maxq=-1), dict(maxq=(1 << 24) + 1), dict(maxl=65), dict(maxl=-1)):
        assert c(**bad) == 2
    for bad in (dict(D=96), dict(g=128), dict(g=16), dict(page=24), dict(page=8)):
        assert c(**bad) == 4
    assert c(B=0, lens=None, table=None) == 0
    assert c(T=0, q=None, out=None) == 0
