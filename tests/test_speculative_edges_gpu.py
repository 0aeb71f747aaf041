"""Calls of the speculative step's operators that lie at the edge of what their documentation allows, on the GPU against
the fp64 oracle (oracle/speculative.py)."""
import numpy as np
import pytest

from oracle import speculative as sp
from test_speculative_gpu import MANY, TOL_TREE, U, dev, dev_cache, f32, ints, np_cache, wide_cache
from weight_quantized_expert_b200 import api

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- probabilities
# The bar is that of test_probs: |err| <= (8 + 2 max|l - max| / temperature) u p, and a step of the subnormal numbers.

def check_probs(x, temp):
    """Out of place, in place, and with logits and probabilities off 16-byte boundaries, alike and unlike each other."""
    import torch
    T, V = x.shape
    want = sp.token_probs(x, temp)
    span = np.where(np.isfinite(x), x.max(-1, keepdims=True).astype(np.float64) - x, 0.0) / temp
    flat, out = torch.zeros(4 + T * V, device="cuda"), torch.zeros(4 + T * V, device="cuda")
    got = [api.focr_token_probs(dev(x), temp)]
    same = dev(x)
    got.append(api.focr_token_probs(same, temp, out=same))
    logits = flat[1:1 + T * V].view(T, V)
    logits.copy_(dev(x))
    got += [api.focr_token_probs(logits, temp, out=out[s:s + T * V].view(T, V)).clone() for s in (1, 2)]
    for g in got:
        g = g.cpu().numpy().astype(np.float64)
        assert not np.isnan(g).any()
        assert (np.abs(g - want) <= (8 + 2 * span) * U * want + 1e-44).all()
        assert (g[np.isneginf(x)] == 0).all()


@pytest.mark.parametrize("V", [1, 3, 5, 10, 100, 777, 1000, 1920, 1921, 10000, 129280])
def test_probs_of_rows_far_below_zero(V):
    # parts of a row that hold no value, or none that is finite, take part in no sum
    rng = np.random.default_rng(V)
    x = 4 * f32(rng, 3, V)
    check_probs(x - np.float32(200), 1.0)
    logp = np.log(sp.token_probs(x)).astype(np.float32)
    check_probs(logp, 0.05)
    check_probs(logp, 1e-6)


@pytest.mark.parametrize("left", [1, 10, 1000])
@pytest.mark.parametrize("T", [1, 60])
def test_probs_of_rows_that_a_mask_leaves_few_tokens_of(left, T):
    rng = np.random.default_rng(left)
    x = np.full((T, 129280), -np.inf, np.float32)
    for t in range(T):
        x[t, rng.choice(129280, left, replace=False)] = -12
    check_probs(x, 0.1)
    x += f32(rng, *x.shape)
    check_probs(x, 0.01)


def test_probs_stay_nan_where_a_row_has_no_distribution():
    for V in (5, 3000, 129280):
        x = np.full((4, V), -np.inf, np.float32)
        x[1, V // 2], x[2, 0], x[3] = np.nan, np.inf, -200
        x[3, 1] = np.nan
        got = api.focr_token_probs(dev(x), 0.5).cpu().numpy()
        assert np.isnan(got[[0, 1, 3]]).all() and np.isnan(got[2]).any()


# ---------------------------------------------------------------- tree attention: what the weights are rounded against
# check_tree's bar, with the largest value among the rows that a node itself sees: |err| <= TOL_TREE max|v seen|.

def values_of(c):
    return sp.values(c[0], c[1]), sp.values(c[2], c[3])


CAPS = [300, MANY]                      # one launch; ranges
LAYOUTS = [(2, 2), (8, 2)]              # up to eight columns of a unit, and more


@pytest.mark.parametrize("hq,hk", LAYOUTS)
@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("factor", [1e4, 1e8, 1e20, 1e30])
def test_a_large_scale_reaches_the_nodes_that_see_its_row_alone(factor, int4, cap, hq, hk):
    # a chain of three behind n = 200 tokens: token 72 is in the ring and seen by none, token 73 by the first node alone
    rng = np.random.default_rng(71)
    B, N, n, R = 3, 3, 200, 300
    q, k, v = f32(rng, B, N, hq, 128), f32(rng, B, N, hk, 128), f32(rng, B, N, hk, 128)
    ref, ring = np_cache(rng, B, hk, R, int4), np_cache(rng, B, hk, 128, int4)
    ring[3][0, :, 72] *= np.float32(factor)
    ring[3][1, :, 73] *= np.float32(factor)
    ring[1][2, :, 72] *= np.float32(factor)
    got = api.focr_rswa_tree(dev(q), dev(k), dev(v), wide_cache(ref, cap), ints([R] * B), dev_cache(ring), ints([n] * B)).cpu().numpy()
    r, g = values_of(ref), values_of(ring)
    want = sp.rswa_tree(q, k, v, r, [R] * B, g, [n] * B)
    for b in range(B):
        for i in range(N):
            seen = [t % 128 for t in range(n + i - 127, n)]
            vmax = max(np.abs(r[1][b]).max(), np.abs(g[1][b][:, seen]).max(), np.abs(v[b, :i + 1]).max())
            assert np.abs(got[b, i] - want[b, i]).max() <= TOL_TREE * vmax, (b, i)


@pytest.mark.parametrize("hq,hk", LAYOUTS)
@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("factor", [1e4, 1e8])
def test_a_large_value_of_no_weight_spares_the_others(factor, int4, cap, hq, hk):
    # all queries lie near one direction, and row 10 against it: its score is about -68, its weight below e^-60
    rng = np.random.default_rng(72)
    B, N, n, R = 2, 3, 50, 300
    way = f32(rng, 128)
    q = way + 0.1 * f32(rng, B, N, hq, 128)
    k, v = f32(rng, B, N, hk, 128), f32(rng, B, N, hk, 128)
    rk, rv = f32(rng, B, hk, R, 128), f32(rng, B, hk, R, 128)
    rk[:, :, 10] = -6 * way
    ref = [*sp.quantise(rk, int4), *sp.quantise(rv, int4)]
    ref[3][:, :, 10] *= np.float32(factor)
    ring = np_cache(rng, B, hk, 128, int4)
    got = api.focr_rswa_tree(dev(q.astype(np.float32)), dev(k), dev(v), wide_cache(ref, cap), ints([R] * B), dev_cache(ring), ints([n] * B)).cpu().numpy()
    r, g = values_of(ref), values_of(ring)
    want = sp.rswa_tree(q.astype(np.float32), k, v, r, [R] * B, g, [n] * B)
    vmax = max(np.abs(np.delete(r[1], 10, 2)).max(), np.abs(g[1]).max(), np.abs(v).max())
    assert np.abs(got - want).max() <= TOL_TREE * vmax


@pytest.mark.parametrize("hq,hk", LAYOUTS)
@pytest.mark.parametrize("R,cap", [(289, 300), (289, MANY), (4096, MANY)])
@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("share,size", [(0.86, 0.1), (0.9, 0.1), (0.9, 0.01), (0.997, 0.003)])
def test_a_key_with_most_of_the_weight_and_a_small_value(share, size, int4, R, cap, hq, hk):
    """A sink.  All other keys have the same score, and all scores are whole numbers, so the bar, relative to an output's norm, is
      digits   each product of a block is off by 0.29 steps of 2^-23 of the largest one (rms), and 64 of them by 8 times that:
               2.8e-7 where the largest one carries the output (the sink's does here);
      scores   the others' common weight is off, relative to the sink's, by the score in log2 x 4 roundings x ln 2 + 2^-22,
               which moves the output by that times (the others' part of it + their share of the weight);
      sums     fp32 roundings of the output and of the weights' sum: 14, and two for each of the blocks that a group of four
               warps (or of the threads that join parts) adds in turn."""
    rng = np.random.default_rng(73)
    B, N, n, top = 1, 3, 64, 7 if int4 else 127
    few = np.arange(16)                  # the dims in which the queries live: all keys but the sink are zero there
    one = np.zeros(128, np.float32)
    one[few] = rng.integers(-126, 127, 16)
    one[3] = 127
    q = np.broadcast_to(one, (B, N, hq, 128)).copy()
    k, v = f32(rng, B, N, hk, 128), f32(rng, B, N, hk, 128)
    k[..., few] = 0
    rk, rv, gk, gv = (f32(rng, B, hk, rows, 128) for rows in (R, R, 128, 128))
    rk[..., few] = gk[..., few] = 0
    sink = R // 3
    rk[:, :, sink] = top * np.sign(one)                # codes of +-top: the row's scale is set below
    ref = [*sp.quantise(rk, int4), *sp.quantise(rv, int4)]
    others = R - 1 + n + 2
    ref[1][:, :, sink] = np.log(share / (1 - share) * others) * np.sqrt(128) / (top * np.abs(one).sum())
    ref[3][:, :, sink] *= np.float32(size)
    ring = [*sp.quantise(gk, int4), *sp.quantise(gv, int4)]
    got = api.focr_rswa_tree(dev(q), dev(k), dev(v), wide_cache(ref, cap), ints([R] * B), dev_cache(ring), ints([n] * B)).cpu().numpy()
    want = sp.rswa_tree(q, k, v, values_of(ref), [R] * B, values_of(ring), [n] * B)
    norm = np.linalg.norm(want, axis=-1)
    rest = np.linalg.norm(want - share * np.repeat(values_of(ref)[1][:, :, sink], hq // hk, 1)[:, None], axis=-1) / norm + 1 - share
    score = np.log2(share / (1 - share) * others) * 4 * U * np.log(2) + 2.0**-22
    bar = 2.8e-7 + score * rest + (14 + 2 * -(-(R + n) // 256)) * U
    assert (np.linalg.norm(got - want, axis=-1) <= bar * norm).all(), (np.linalg.norm(got - want, axis=-1) / norm / bar).max()


# ---------------------------------------------------------------- cache writes

@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("what", [np.nan, np.inf, -np.inf])
def test_a_row_with_what_is_no_number_is_written_as_such(what, int4):
    import torch
    rng = np.random.default_rng(81)
    rows, heads = 40, 2
    k, v = f32(rng, rows, heads, 128), f32(rng, rows, heads, 128)
    want = [np.zeros((1, heads, rows, 64 if int4 else 128), np.uint8 if int4 else np.int8), np.zeros((1, heads, rows), np.float32)] * 2
    want = [x.copy() for x in want]
    sp.kv_write(want, k, v, [rows], [0], n_max=rows)
    for i, x, codes, scale in ((3, k, *want[:2]), (17, k, *want[:2]), (17, v, *want[2:]), (39, v, *want[2:])):
        x[i, 1, (7 * i) % 128] = what
        codes[0, 1, i], scale[0, 1, i] = 0, abs(what)
    cache = api.new_kv_cache(1, heads, rows, api.W_INT4 if int4 else api.W_INT8)
    api.focr_kv_write(cache, dev(k), dev(v), ints([rows]), ints([0]))
    torch.cuda.synchronize()
    for got, x in zip(cache, want):
        np.testing.assert_array_equal(got.cpu().numpy(), x)
    for got, bad in zip(api.focr_kv_read(cache, ints([rows])), ([3, 17], [17, 39])):
        nan = np.isnan(got.cpu().numpy()[0])
        assert nan[1, bad].all() and nan.sum() == 2 * 128
    # rows 0 .. 2 are fine; row 3 is seen by the second sequence
    two = [torch.cat((x, x)) for x in cache]
    q = dev(f32(rng, 2, 1, heads, 128))
    ring = api.new_kv_cache(2, heads, 128, api.W_INT4 if int4 else api.W_INT8)
    out = api.focr_rswa_tree(q, q, q, two, ints([3, 4]), ring, ints([0, 0]))
    assert out[1, 0, 1].isnan().all() and out.isfinite().sum().item() == 3 * 128


def test_a_flat_ragged_prompt_is_written_whole_by_default():
    # offsets and counts alone: a sequence may have more than its share of the rows
    import torch
    rng = np.random.default_rng(82)
    k, v = f32(rng, 50, 2, 128), f32(rng, 50, 2, 128)
    want = np_cache(rng, 3, 2, 64, False)
    cache = dev_cache(want)
    count, row0 = [40, 1, 9], [0, 40, 41]
    api.focr_kv_write(cache, dev(k), dev(v), ints(count), ints([0, 5, 55]), row0=ints(row0))
    sp.kv_write(want, k, v, count, [0, 5, 55], row0, n_max=50)
    torch.cuda.synchronize()
    for got, x in zip(cache, want):
        np.testing.assert_array_equal(got.cpu().numpy(), x)


# ---------------------------------------------------------------- consecutive steps

def test_consecutive_steps_attend_over_what_the_ones_before_committed():
    """Three steps as the header puts them together: the sampled token is node 0 of the next tree, [0, path + 1] is committed,
    n_gen advances by n_accept + 1.  Each token's attention is checked against the plain formula over the sequence of committed
    tokens (no tree, no ring): positions P - 127 .. P, the rows of earlier steps as the quantiser leaves them.  Then the same
    from a captured step, replayed."""
    import torch
    rng = np.random.default_rng(91)
    B, D, heads, V, R, S = 3, 6, 4, 12, 100, 3
    N, G = D + 1, heads * 128
    parent = [-1, -1, 0, 0, 1, 2]
    nodes = [-1] + [p + 1 for p in parent]
    depth = [len(x) - 1 for x in sp.tree_lines(nodes)]
    first, ref_len = [126, 0, 300], [100, 0, 37]
    tables = [dev(f32(rng, V, G)) for _ in range(3)]
    head = dev(0.3 * f32(rng, G, V))
    prompt, old = [f32(rng, B * R, heads, 128) for _ in range(2)], [f32(rng, B * 300, heads, 128) for _ in range(2)]
    drafts = rng.integers(0, V, (S, B, D)).astype(np.int32)
    u = rng.random((S, B, D + 1), np.float32)
    u[:, 0, [0, 2]], u[:, 2, :D] = 0.0, 0.999          # the first sequence accepts drafts 0 and 2, the last one few or none
    x_first = rng.integers(0, V, B).astype(np.int32)
    ref, ring = api.new_kv_cache(B, heads, R), api.new_kv_cache(B, heads, 128)
    api.focr_kv_write(ref, dev(prompt[0]), dev(prompt[1]), ints(ref_len), ints([0] * B), n_max=R)
    api.focr_kv_write(ring, dev(old[0]), dev(old[1]), ints(first), ints([0] * B), n_max=300, wrap=True)
    start = [x.clone() for x in ring]
    x, n, d_drafts, d_u = ints(x_first), ints(first), dev(drafts[0]), dev(u[0])
    d_depth, d_nodes, d_parent, d_len = ints(depth), ints([nodes] * B), ints([parent] * B), ints(ref_len)

    def step():
        toks = torch.cat((x[:, None], d_drafts), 1)
        q, k, v = (t[toks.long()].view(B * N, heads, 128) for t in tables)
        q, k = api.focr_qk_norm_rope(q, k, (n[:, None] + d_depth).view(-1), norm=True)
        shape = (B, N, heads, 128)
        out = api.focr_rswa_tree(q.view(shape), k.view(shape), v.view(shape), ref, d_len, ring, n, d_nodes)
        probs = api.focr_token_probs(out.view(B * N, G) @ head, 0.9).view(B, N, V)
        taken, path, nxt = api.focr_spec_verify(probs, None, d_drafts, d_parent, None, d_u)
        index = torch.cat((torch.zeros_like(x)[:, None], path + 1), 1)
        api.focr_kv_write(ring, k, v, taken + 1, n, index=index, n_max=N, wrap=True)
        n.add_(taken + 1)
        x.copy_(nxt)
        return dict(q=q, k=k, v=v, out=out, probs=probs, taken=taken, path=path, next=nxt, n=n, x=x)

    def steps(one):
        for t, y in zip(ring, start):
            t.copy_(y)
        x.copy_(ints(x_first))
        n.copy_(ints(first))
        got = []
        for s in range(S):
            d_drafts.copy_(dev(drafts[s]))
            d_u.copy_(dev(u[s]))
            got.append({name: t.clone().cpu().numpy() for name, t in one().items()})
        return got

    got = steps(step)
    rows = lambda t: sp.values(*sp.quantise(t, False))  # noqa: E731
    r = [rows(t.reshape(B, R, heads, 128)) for t in prompt]
    seqs = [[[list(rows(t.reshape(B, 300, heads, 128)[b, :first[b]])) for t in old], int(x_first[b])] for b in range(B)]
    for s, g in enumerate(got):
        want = sp.spec_verify(g["probs"], None, drafts[s], np.array([parent] * B), None, u[s])
        for name, w in zip(("taken", "path", "next"), want):
            np.testing.assert_array_equal(g[name], w)
        lines = sp.tree_lines(nodes)
        for b, seq in enumerate(seqs):
            kv, tok = seq
            P = len(kv[0])
            q, k, v, out = (g[name].reshape(B, N, heads, 128)[b] for name in ("q", "k", "v", "out"))
            at = sp.qk_norm_rope(tables[1].cpu().numpy()[np.r_[tok, drafts[s, b]]].reshape(N, heads, 128), [P + d for d in depth], norm=True)
            assert np.abs(k - at).max() <= 2e-5            # the sampled token and the drafts, at their positions
            for i, line in enumerate(lines):
                line = line[::-1]
                keys, vals = ([*np.asarray(c)[:], *y[line]] for c, y in zip(kv, (k, v)))
                keys, vals = keys[-128:], vals[-128:]
                for h in range(heads):
                    kk = np.array([*r[0][b, :ref_len[b], h], *[z[h] for z in keys]], np.float64)
                    vv = np.array([*r[1][b, :ref_len[b], h], *[z[h] for z in vals]], np.float64)
                    w = kk @ q[i, h].astype(np.float64) / np.sqrt(128)
                    w = np.exp(w - w.max())
                    assert np.abs(out[i, h] - w @ vv / w.sum()).max() <= TOL_TREE * np.abs(vv).max(), (s, b, i, h)
            done = [0, *(g["path"][b, :g["taken"][b]] + 1)]
            for c, y in zip(kv, (k, v)):
                c += list(rows(np.ascontiguousarray(y[done])))
            seq[1] = int(g["next"][b])
            assert g["n"][b] == len(kv[0]) and g["x"][b] == seq[1]
        assert g["taken"][0] >= 2
    final = [t.clone() for t in ring]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()

    def replay():
        graph.replay()
        return held

    for a, b in zip(got, steps(replay)):
        for name in a:
            np.testing.assert_array_equal(a[name], b[name], err_msg=name)
    for a, b in zip(final, ring):
        assert torch.equal(a, b)
