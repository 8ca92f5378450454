"""The calls that keep a cache within a budget, without a GPU: the refusals that
are made before anything is launched."""
import ctypes

import pytest
import torch

from paged_kv_cache_06_gb300 import ops

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
FAKE = 0x100000       # aligned, non-null; never dereferenced by these calls
FAR = 0x10000000
ODD = 0x100008        # not 16-byte aligned


def P(x):
    return ctypes.c_void_p(x) if x else None


def norm(**kw):
    a = dict(q_out=FAR, k=FAKE, v=FAKE, ks=0, vs=0, bt=FAKE, sl=FAKE, qs=FAKE, rp=0, rates=FAKE, q=FAKE, kn=FAKE,
             vn=FAKE, qw=FAKE, kw=FAKE, eps=1e-6, sq=1536, sk=256, sv=256, rows=4, total=9, hq=12, hk=2, d=128,
             rot=128, layout=0, m=1.0, bs=16, mbpr=16, nb=64, msl=200)
    a.update(kw)
    return ops.lib().paged_kv_norm_rope_append(
        *[P(a[n]) for n in ("q_out", "k", "v", "ks", "vs", "bt", "sl", "qs", "rp", "rates", "q", "kn", "vn", "qw", "kw")],
        a["eps"], a["sq"], a["sk"], a["sv"], a["rows"], a["total"], a["hq"], a["hk"], a["d"], a["rot"], a["layout"],
        a["m"], a["bs"], a["mbpr"], a["nb"], a["msl"], None, None)


def test_norm_rope_append_refusals():
    for n in ("k", "v", "bt", "sl", "qs", "rates", "q", "kn", "vn", "q_out", "qw", "kw"):
        assert norm(**{n: 0}) == INVALID, n
    for n in ("k", "v", "q", "kn", "vn", "q_out", "qw", "kw"):
        assert norm(**{n: ODD}) == INVALID, n
    for eps in (-1e-6, float("nan"), float("inf")):
        assert norm(eps=eps) == INVALID
    assert norm(ks=FAKE) == INVALID and norm(layout=2) == INVALID and norm(m=float("inf")) == INVALID
    assert norm(d=120, rot=112) == UNSUPPORTED                        # a multiple of 8, as rope_append takes
    assert norm(d=528, rot=128, sq=1 << 20, sk=1 << 20, sv=1 << 20) == UNSUPPORTED
    assert norm(rot=24) == UNSUPPORTED and norm(rot=144) == INVALID
    size = 9 * 12 * 128 * 2
    for n in ("qw", "kw"):                                            # the output over a weight
        assert norm(**{n: FAR}) == INVALID and norm(**{n: FAR + size - 16}) == INVALID
    assert norm(q=FAR + 256) == INVALID and norm(q_out=FAKE, sq=1544) == INVALID
    assert norm(rows=0, k=0) == 0 and norm(total=0, q=0) == 0


def decode(**kw):
    a = dict(out=FAR, w=2 * FAR, q=FAKE, k=FAKE, v=FAKE, ks=0, vs=0, bt=FAKE, sl=FAKE, rows=4, hq=12, hk=2, d=128, bs=16,
             scale=0.1, mbpr=16, nb=64, msl=200, stride=200, ws=3 * FAR, wsb=None)
    a.update(kw)
    if a["wsb"] is None:
        a["wsb"] = ops.decode_weights_workspace_size(4, 12, 2, 128, 200, 16)
    return ops.lib().paged_attention_decode_weights(
        *[P(a[n]) for n in ("out", "w", "q", "k", "v", "ks", "vs", "bt", "sl")], a["rows"], a["hq"], a["hk"], a["d"],
        a["bs"], a["scale"], a["mbpr"], a["nb"], a["msl"], a["stride"], P(a["ws"]), a["wsb"], None, None)


def test_decode_weights_refusals():
    for n in ("out", "w", "q", "k", "v", "bt", "sl"):
        assert decode(**{n: 0}) == INVALID, n
    for n in ("out", "q", "k", "v"):
        assert decode(**{n: ODD}) == INVALID, n
    assert decode(ks=FAKE) == INVALID and decode(vs=FAKE) == INVALID
    assert decode(stride=199) == INVALID and decode(msl=257, stride=300) == INVALID
    assert decode(scale=float("nan")) == INVALID and decode(hq=12, hk=5) == INVALID and decode(bs=0) == INVALID
    assert decode(d=64) == UNSUPPORTED and decode(bs=24) == UNSUPPORTED and decode(rows=1025) == UNSUPPORTED
    assert decode(hq=18, hk=2) == UNSUPPORTED and decode(nb=1 << 27) == UNSUPPORTED
    assert decode(ws=0) == WORKSPACE and decode(wsb=64) == WORKSPACE and decode(ws=3 * FAR + 16) == WORKSPACE
    for n in ("out", "q", "ws"):                                      # the sums over what is read or written
        at = {"out": FAR, "q": FAKE, "ws": 3 * FAR}[n]
        assert decode(w=at) == INVALID and decode(w=at - 4 * 2 * 200 * 4 + 4) == INVALID, n
    assert decode(q=FAR) == INVALID and decode(ws=FAR) == INVALID         # the output over what is read or written
    assert decode(rows=0, q=0) == 0


def test_decode_weights_workspace_size_host_arithmetic():
    n = ops.decode_weights_workspace_size(4, 12, 2, 128, 200, 16)
    assert n % 256 == 0 and n >= 4 * 2 * 200 * 6 * 4
    for bad in ((0, 12, 2, 128, 200, 16), (4, 12, 5, 128, 200, 16), (4, 12, 2, 64, 200, 16), (4, 18, 2, 128, 200, 16),
                (4, 12, 2, 128, -1, 16), (4, 12, 2, 128, 200, 24), (1025, 12, 2, 128, 200, 16)):
        assert ops.decode_weights_workspace_size(*bad) == 0, bad


def test_decode_weights_sizes_that_are_refused_have_no_workspace():
    for kw in (dict(rows=1024, hk=1024, hq=1024, msl=1 << 16, mbpr=1 << 12, stride=1 << 16), dict(bs=1040), dict(bs=4096)):
        a = dict(rows=4, hq=12, hk=2, d=128, msl=200, bs=16)
        a.update({n: x for n, x in kw.items() if n in a})
        assert ops.decode_weights_workspace_size(a["rows"], a["hq"], a["hk"], a["d"], a["msl"], a["bs"]) == 0, kw
        assert decode(w=1 << 60, wsb=1 << 62, **kw) in (INVALID, UNSUPPORTED), kw
    most = (1024, 1024, 1024, 128, 32640, 16)                         # 2^31 granules less 2^23
    assert ops.decode_weights_workspace_size(*most) > 0
    assert ops.decode_weights_workspace_size(*most[:4], 32768, 16) == 0


def prefill(**kw):
    a = dict(w=2 * FAR, q=FAR, k=FAKE, ks=0, bt=FAKE, sl=FAKE, qs=FAKE, rows=4, total=90, hq=12, hk=2, d=128, bs=16,
             scale=0.1, window=32, mbpr=16, nb=64, msl=200, stride=200, ws=3 * FAR, wsb=None)
    a.update(kw)
    if a["wsb"] is None:
        a["wsb"] = ops.prefill_weights_workspace_size(4, 90, 12, 2, 128, 200, 16, window=32)
    return ops.lib().paged_attention_prefill_weights(
        *[P(a[n]) for n in ("w", "q", "k", "ks", "bt", "sl", "qs")], a["rows"], a["total"], a["hq"], a["hk"], a["d"],
        a["bs"], a["scale"], a["window"], a["mbpr"], a["nb"], a["msl"], a["stride"], P(a["ws"]), a["wsb"], None, None)


def test_prefill_weights_refusals():
    for n in ("w", "q", "k", "bt", "sl", "qs"):
        assert prefill(**{n: 0}) == INVALID, n
    assert prefill(q=ODD) == INVALID and prefill(k=ODD) == INVALID
    assert prefill(window=0) == INVALID and prefill(window=-1) == INVALID
    assert prefill(stride=199) == INVALID and prefill(msl=257, stride=300) == INVALID
    assert prefill(scale=float("inf")) == INVALID and prefill(hq=12, hk=5) == INVALID and prefill(nb=0) == INVALID
    assert prefill(d=64) == UNSUPPORTED and prefill(bs=24) == UNSUPPORTED and prefill(rows=1025) == UNSUPPORTED
    assert prefill(hq=129, hk=1) == UNSUPPORTED and prefill(nb=1 << 27) == UNSUPPORTED
    assert prefill(total=1 << 30, msl=1 << 20, stride=1 << 20, mbpr=1 << 17, window=1 << 30) == UNSUPPORTED


def test_prefill_weights_workspace():
    n = ops.prefill_weights_workspace_size(4, 90, 12, 2, 128, 200, 16)
    assert n > 0 and n % 256 == 0
    assert ops.prefill_weights_workspace_size(4, 9000, 12, 2, 128, 200, 16, window=1) <= \
        ops.prefill_weights_workspace_size(4, 9000, 12, 2, 128, 200, 16, window=32) < \
        ops.prefill_weights_workspace_size(4, 9000, 12, 2, 128, 200, 16)
    for bad in ((0, 90, 12, 2, 128, 200, 16), (4, -1, 12, 2, 128, 200, 16), (4, 90, 12, 5, 128, 200, 16),
                (4, 90, 12, 2, 64, 200, 16), (4, 90, 12, 2, 128, 200, 24), (4, 90, 129, 1, 128, 200, 16)):
        assert ops.prefill_weights_workspace_size(*bad) == 0, bad
    assert ops.prefill_weights_workspace_size(4, 90, 12, 2, 128, 200, 16, window=0) == 0
    assert prefill(rows=0, q=0) == 0 and prefill(total=0, q=0) == 0


@pytest.mark.gpu
def test_prefill_weights_workspace_refusals_of_a_device(cuda_device):
    """(The size depends on the device's SMs.)"""
    assert prefill(ws=0) == WORKSPACE and prefill(wsb=256) == WORKSPACE and prefill(ws=3 * FAR + 16) == WORKSPACE
    for at in (FAR, 3 * FAR):                                          # the sums over what is read or written
        assert prefill(w=at) == INVALID and prefill(w=at - 4 * 2 * 200 * 4 + 4) == INVALID
    assert prefill(q=3 * FAR) == INVALID


def evict(**kw):
    a = dict(k=FAKE, v=FAKE, bt=FAKE, sl=FAKE, w=FAR, pos=2 * FAR, tr=FAKE, nx=FAKE, wo=None, po=None, new=3 * FAR,
             layers=2, rows=4, hk=2, d=128, eb=2, bs=16, mbpr=16, nb=64, msl=200, stride=200, budget=100, sinks=4,
             recent=20)
    a.update(kw)
    a["wo"], a["po"] = a["w"] if a["wo"] is None else a["wo"], a["pos"] if a["po"] is None else a["po"]
    return ops.lib().paged_kv_evict(
        *[P(a[n]) for n in ("k", "v", "bt", "sl", "w", "pos", "tr", "nx", "wo", "po", "new")], a["layers"], a["rows"],
        a["hk"], a["d"], a["eb"], a["bs"], a["mbpr"], a["nb"], a["msl"], a["stride"], a["budget"], a["sinks"],
        a["recent"], None, None)


def test_evict_refusals():
    for n in ("k", "v", "bt", "sl", "w", "pos"):
        assert evict(**{n: 0}) == INVALID, n
    assert evict(k=ODD) == INVALID and evict(v=ODD) == INVALID
    assert evict(budget=0) == INVALID and evict(sinks=-1) == INVALID and evict(recent=-1) == INVALID
    assert evict(sinks=50, recent=51) == INVALID and evict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1) == INVALID
    assert evict(stride=199) == INVALID and evict(msl=257, stride=300) == INVALID
    assert evict(eb=4) == INVALID and evict(d=12) == UNSUPPORTED and evict(d=8, eb=1) == UNSUPPORTED
    assert evict(msl=196609, stride=196609, mbpr=20000) == UNSUPPORTED and evict(nb=1 << 27) == UNSUPPORTED
    assert evict(rows=-1) == INVALID and evict(layers=-1) == INVALID and evict(hk=0) == INVALID
    assert evict(rows=0, k=0) == 0 and evict(layers=0, k=0) == 0


def test_evict_outputs_lie_over_nothing_else():
    wide = 2 * 4 * 2 * 200 * 4
    out, pos = 4 * FAR, 5 * FAR
    assert evict(wo=out) == INVALID and evict(po=pos) == INVALID       # in place both, or neither
    for x in (2 * FAR, FAR + 4, FAR - wide + 4, 3 * FAR, pos):         # token_pos, part of weights, new lengths, positions
        assert evict(wo=x, po=pos) == INVALID, x
    for x in (FAR, 2 * FAR + 4, 2 * FAR - wide + 4, 3 * FAR, out):
        assert evict(wo=out, po=x) == INVALID, x
    for n, size in (("sl", 16), ("bt", 256), ("tr", 16), ("nx", 16), ("w", wide), ("pos", wide)):
        at = {"w": FAR, "pos": 2 * FAR}.get(n, FAKE)
        assert evict(new=at) == INVALID and evict(new=at + size - 4) == INVALID, n
    assert evict(wo=FAKE, po=pos) == INVALID and evict(wo=out, po=FAKE + 12) == INVALID


def test_evict_outputs_lie_over_no_pool():
    size = 2 * 64 * 16 * 2 * 128 * 2
    out, pos, far = 4 * FAR, 5 * FAR, 6 * FAR
    for n in ("k", "v"):
        for x in (far, far + size - 4):
            assert evict(**{n: far}, new=x) == INVALID, n
            assert evict(**{n: far}, w=x) == INVALID and evict(**{n: far}, pos=x) == INVALID, n          # in place
            assert evict(**{n: far}, wo=x, po=pos) == INVALID and evict(**{n: far}, wo=out, po=x) == INVALID, n
    # sizes whose product passes 64 bits
    huge = dict(layers=60000, nb=1 << 20, hk=1 << 12, d=1 << 19, pos=1 << 43, w=1 << 42)
    assert evict(k=far, v=1 << 45, **huge) == INVALID


def test_weights_hooks_refusals():
    for bad in ((-1, 0, 0), (0, -1, 0), (0, 4, 0), (0, 0, -1)):
        assert ops.lib().pkv_debug_set_weights_hooks(*bad) == INVALID, bad
    ops.debug_set_weights_hooks(3, "sums", 5)
    ops.debug_set_weights_hooks()


def test_ops_refuse_cpu_tensors_and_wrong_shapes():
    h, i = torch.zeros(4, 12, 128, dtype=torch.float16), torch.zeros(4, dtype=torch.int32)
    pool = torch.zeros(4, 16, 2, 128, dtype=torch.float16)
    bt, qs = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(5, dtype=torch.int32)
    rates, w = torch.zeros(64, dtype=torch.int64), torch.zeros(128, dtype=torch.float16)
    with pytest.raises(ValueError):
        ops.norm_rope_append(pool, pool, bt, i, qs, h[:, :2], h[:, :2], rates, w, 16)
    with pytest.raises(ValueError):
        ops.norm_rope_append(pool, pool, bt, i, qs, h, h, rates, w, 16, layout="whole")
    with pytest.raises(ValueError):
        ops.evict(pool, pool, bt, i, torch.zeros(4, 2, 32), torch.zeros(4, 2, 32, dtype=torch.int32), 8, 32)
