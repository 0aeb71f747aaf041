"""The speculative step's entry points refuse bad arguments before anything is launched (no GPU needed)."""
import ctypes

import pytest

from weight_quantized_expert_b200 import api

INVALID, UNSUPPORTED = 1, 2
_buf = (ctypes.c_float * (1 << 16))()
A = (ctypes.addressof(_buf) + 255) // 256 * 256     # a 256-byte aligned address that nothing dereferences


def at(i):
    return A + 4096 * i


def cache(type=api.W_INT8, B=1, heads=10, cap=128, k=at(0), ks=at(1), v=at(2), vs=at(3)):
    return api.KVCacheDesc(k, ks, v, vs, type, B, heads, cap)


ROPE = dict(q=at(0), ldq=1280, hq=10, k=at(8), ldk=1280, hk=10, pos=at(1), T=1, gq=None, gk=None, eps=1e-6, theta=1e4,
            rot=128, flags=0, qo=at(2), ldqo=1280, ko=at(10), ldko=1280)


def rope(**kw):
    a = dict(ROPE, **kw)
    return api.lib().focr_qk_norm_rope(*a.values(), None)


@pytest.mark.parametrize("bad,status,word", [
    (dict(q=None), INVALID, "NULL"), (dict(pos=None), INVALID, "NULL"), (dict(ko=None), INVALID, "NULL"),
    (dict(T=0), INVALID, "T="), (dict(T=api.T_MAX + 1), INVALID, "T="), (dict(hq=0), INVALID, "heads"),
    (dict(hk=129), INVALID, "heads"), (dict(rot=3), UNSUPPORTED, "rot_dim"), (dict(rot=130), UNSUPPORTED, "rot_dim"),
    (dict(rot=0), UNSUPPORTED, "rot_dim"), (dict(flags=4), INVALID, "flags"), (dict(theta=0.0), INVALID, "theta"),
    (dict(theta=float("inf")), INVALID, "theta"), (dict(eps=-1.0), INVALID, "eps"), (dict(eps=float("nan")), INVALID, "eps"),
    (dict(ldq=1276), INVALID, "stride"), (dict(ldko=1282), INVALID, "stride"), (dict(q=at(0) + 4), INVALID, "aligned"),
    (dict(gq=at(4) + 8), INVALID, "aligned"), (dict(pos=at(1) + 2), INVALID, "positions"),
    (dict(qo=at(0) + 16), INVALID, "overlap"), (dict(ko=at(0)), INVALID, "overlap"), (dict(qo=at(10)), INVALID, "overlap"),
    (dict(T=2, qo=at(0), ldqo=2560), INVALID, "overlap"),
])
def test_rope_refusals(bad, status, word):
    assert rope(**bad) == status and word in api.focr_last_error()


WRITE = dict(k=at(8), ldk=1280, v=at(20), ldv=1280, rows=4, row0=None, count=at(4), index=None, n_max=4, start=at(5), flags=0)


def write(c=None, **kw):
    a = dict(WRITE, **kw)
    c = cache() if c is None else c
    return api.lib().focr_kv_write(ctypes.byref(c), *a.values(), None)


@pytest.mark.parametrize("c,status,word", [
    (dict(k=None), INVALID, "NULL"), (dict(vs=None), INVALID, "NULL"), (dict(type=api.W_BF16), UNSUPPORTED, "type"),
    (dict(B=0), INVALID, "sequences"), (dict(heads=0), INVALID, "heads"), (dict(cap=40000), INVALID, "rows"),
    (dict(v=at(2) + 8), INVALID, "aligned"), (dict(ks=at(1) + 2), INVALID, "aligned"),
])
def test_cache_refusals(c, status, word):
    assert write(cache(**c)) == status and word in api.focr_last_error()
    d = cache(**c)
    assert api.lib().focr_kv_read(ctypes.byref(d), at(4), at(5), at(40), None) == status


@pytest.mark.parametrize("bad,word", [
    (dict(k=None), "NULL"), (dict(count=None), "NULL"), (dict(start=None), "NULL"), (dict(flags=2), "flags"),
    (dict(n_max=0), "n_max"), (dict(n_max=32769), "n_max"), (dict(rows=0), "n_rows"), (dict(ldk=1276), "stride"),
    (dict(ldv=1281), "stride"), (dict(v=at(20) + 4), "aligned"), (dict(index=at(6) + 1), "misaligned"),
])
def test_write_refusals(bad, word):
    assert write(**bad) == INVALID and word in api.focr_last_error()
    assert api.lib().focr_kv_write(None, *WRITE.values(), None) == INVALID


def test_read_refusals():
    L, c = api.lib(), cache(cap=1, heads=1)
    assert L.focr_kv_read(None, at(4), at(5), at(6), None) == INVALID
    for args, word in (((None, at(5), at(6)), "NULL"), ((at(4), None, at(6)), "NULL"), ((at(4), at(5) + 4, at(6)), "misaligned"),
                       ((at(4), at(5), at(5) + 16), "overlap")):
        assert L.focr_kv_read(ctypes.byref(c), *args, None) == INVALID and word in api.focr_last_error()


def tree(ref=None, ring=None, **kw):
    a = dict(dict(q=at(8), k=at(10), v=at(12), B=1, N=1, hq=10), **{k: kw.pop(k) for k in ("q", "k", "v", "B", "N", "hq") if k in kw})
    b = dict(dict(n_gen=at(5), parent=None, n_nodes=None, out=at(14), ws=None, ws_bytes=0),
             **{k: kw.pop(k) for k in ("n_gen", "parent", "n_nodes", "out", "ws", "ws_bytes") if k in kw})
    ref, ring = cache(**(ref or dict(cap=289))), cache(**(ring or {}))
    return api.lib().focr_rswa_tree(*a.values(), ctypes.byref(ref), kw.get("ref_len", at(4)), ctypes.byref(ring), *b.values(), None)


@pytest.mark.parametrize("bad,status,word", [
    (dict(q=None), INVALID, "NULL"), (dict(ref_len=None), INVALID, "NULL"), (dict(out=None), INVALID, "NULL"),
    (dict(ref=dict(type=api.W_INT4)), UNSUPPORTED, "one type"), (dict(ring=dict(cap=64)), UNSUPPORTED, "slots"),
    (dict(ring=dict(B=2)), INVALID, "sequences"), (dict(ring=dict(heads=5)), INVALID, "heads"), (dict(B=2), INVALID, "sequences"),
    (dict(hq=15), UNSUPPORTED, "query heads"), (dict(hq=5), UNSUPPORTED, "query heads"), (dict(hq=130), UNSUPPORTED, "query heads"),
    (dict(N=0), INVALID, "nodes"), (dict(N=65), INVALID, "nodes"), (dict(N=33, hq=20), INVALID, "nodes"),
    (dict(N=1 << 30, hq=40), INVALID, "nodes"), (dict(q=at(8) + 4), INVALID, "aligned"), (dict(parent=at(6) + 2), INVALID, "misaligned"),
    (dict(ref=dict(cap=32768)), INVALID, "workspace"), (dict(ref=dict(cap=32768), ws=at(15), ws_bytes=256), INVALID, "workspace"),
    (dict(ref=dict(cap=32768), ws=at(15) + 64, ws_bytes=1 << 30), INVALID, "workspace"),
    (dict(out=at(8)), INVALID, "overlap"), (dict(out=at(10)), INVALID, "overlap"), (dict(out=at(12) + 16), INVALID, "overlap"),
])
def test_tree_refusals(bad, status, word):
    assert tree(**bad) == status and word in api.focr_last_error()


def test_tree_workspace_sizes():
    size = api.focr_rswa_tree_workspace_bytes
    assert size(1, 1, 10, 10, 289) == 0 and size(8, 32, 10, 10, 32768) % 256 == 0 < size(8, 32, 10, 10, 32768)
    assert all(size(*a) == 0 for a in ((0, 1, 1, 1, 64), (1, 0, 1, 1, 64), (1, 1, 1, 0, 64), (1, 1, 1, 2, 64), (1, 1, 1, 1, 1 << 20)))


@pytest.mark.parametrize("args,word", [
    ((None, 1, 8, 1.0, at(1)), "NULL"), ((at(0), 0, 8, 1.0, at(1)), "T="), ((at(0), 1, 0, 1.0, at(1)), "V="),
    ((at(0), 1, (1 << 20) + 1, 1.0, at(1)), "V="), ((at(0), 1, 8, 0.0, at(1)), "temperature"),
    ((at(0), 1, 8, 1e-7, at(1)), "temperature"), ((at(0), 1, 8, float("nan"), at(1)), "temperature"), ((at(0), 1, 8, float("inf"), at(1)), "temperature"),
    ((at(0) + 2, 1, 8, 1.0, at(1)), "misaligned"), ((at(0), 1, 8, 1.0, at(0) + 4), "overlap"),
])
def test_probs_refusals(args, word):
    assert api.lib().focr_token_probs(*args, None) == INVALID and word in api.focr_last_error()


VERIFY = dict(target=at(0), draft=at(2), V=8, tokens=at(4), parent=at(5), n_nodes=at(6), u=at(7), B=1, N=4, n_accept=at(8),
              path=at(9), next=at(10))


@pytest.mark.parametrize("bad,word", [
    (dict(target=None), "NULL"), (dict(tokens=None), "NULL"), (dict(u=None), "NULL"), (dict(next=None), "NULL"),
    (dict(B=0), "B="), (dict(B=5000), "B="), (dict(N=0), "N="), (dict(N=65), "N="), (dict(V=0), "V="),
    (dict(V=(1 << 20) + 1), "V="), (dict(draft=at(2) + 1), "misaligned"), (dict(path=at(9) + 2), "misaligned"),
])
def test_verify_refusals(bad, word):
    assert api.lib().focr_spec_verify(*dict(VERIFY, **bad).values(), None) == INVALID and word in api.focr_last_error()


def test_the_binding_refuses_cpu_tensors_and_wrong_shapes():
    import torch
    q = torch.zeros(1, 10, 128)
    c = api.new_kv_cache(1, 10, 128, api.W_INT8, device="cpu")
    one = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: api.focr_qk_norm_rope(q, q, one), lambda: api.focr_kv_write(c, q, q, one, one),
                 lambda: api.focr_kv_read(c, one), lambda: api.focr_rswa_tree(q[None], q[None], q[None], c, one, c, one),
                 lambda: api.focr_token_probs(q), lambda: api.focr_spec_verify(q, None, one, None, None, q),
                 lambda: api.new_kv_cache(1, 1, 1, api.W_BF16, device="cpu")):
        with pytest.raises(api.FocrError):
            call()


SMALL = dict(heads=1, cap=8)    # 1 KB of codes, 32 B of scales: the default addresses are apart


@pytest.mark.parametrize("c,bad", [
    (dict(ks=at(0) + 512), {}), (dict(v=at(0) + 1008), {}), (dict(vs=at(1) + 28), {}), ({}, dict(k=at(0))), ({}, dict(v=at(3) - 512)),
    ({}, dict(count=at(1))), ({}, dict(start=at(0) + 1020)), ({}, dict(index=at(2))), ({}, dict(row0=at(3))),
])
def test_write_refuses_overlapping_buffers(c, bad):
    assert write(cache(**SMALL, **c), **bad) == INVALID and "overlap" in api.focr_last_error()


@pytest.mark.parametrize("args", [(at(4), at(0), at(6)), (at(4), at(5), at(3) - 16), (at(5) + 16, at(5), at(6)), (at(4), at(5), at(0) + 1008)])
def test_read_refuses_overlapping_buffers(args):
    c = cache(**SMALL)
    assert api.lib().focr_kv_read(ctypes.byref(c), *args, None) == INVALID and "overlap" in api.focr_last_error()


@pytest.mark.parametrize("bad", [
    dict(out=at(4)), dict(out=at(5)), dict(out=at(0)), dict(out=at(6), parent=at(7)), dict(out=at(6), n_nodes=at(6) + 64),
    dict(ref=dict(cap=32768), ws=at(8), ws_bytes=1 << 30), dict(ref=dict(cap=32768), ws=at(14), ws_bytes=1 << 30),
])
def test_tree_refuses_overlapping_buffers(bad):
    assert tree(**bad) == INVALID and "overlap" in api.focr_last_error()


@pytest.mark.parametrize("bad", [dict(qo=at(1)), dict(ko=at(1)), dict(gq=at(3)), dict(gk=at(11))])
def test_rope_refuses_outputs_over_positions_and_weights(bad):
    assert rope(**bad) == INVALID and "overlap" in api.focr_last_error()


@pytest.mark.parametrize("bad", [dict(path=at(4)), dict(next=at(8)), dict(n_accept=at(9) + 12), dict(n_accept=at(7) + 16),
                                 dict(path=at(0) + 144), dict(next=at(2)), dict(path=at(5)), dict(next=at(6))])
def test_verify_refuses_overlapping_buffers(bad):
    assert api.lib().focr_spec_verify(*dict(VERIFY, **bad).values(), None) == INVALID and "overlap" in api.focr_last_error()
