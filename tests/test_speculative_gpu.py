"""The speculative step's operators on the GPU against the fp64 oracle (oracle/speculative.py).

Tolerances (derived before the first run; u = 2^-24, half a step of fp32):
  rotation   |err| <= 3e-6 max|y|: the norm costs a few u per value (sum of 128 squares in a tree, root, quotient, two
             products: < 12 u = 7e-7), the angle 2^-25 revolutions (2e-7 rad) and sincos < 4 u, each times the two
             values of a pair, and the pair's two products and sum 3 u.
  tree       the output is a convex combination of value rows, so |err| <= 2 (relative error of a weight) max|v|.  A
             weight exp(s) is off by the absolute error of s plus a few u.  s = q.k / sqrt(128) is off by at most
             sum|q||k| 2^-22 / sqrt(128): 128 products of values below 4.5 are < 60 x 2^-22 = 1.5e-5 in the worst case.
             3e-5 max|v| holds it (the bar of the fp32 decode attention).
  probs      |err| <= (8 + 2 max|l - max| / temperature) u p: the quotient's rounding is magnified by its size, exp
             2 u, the sum's tree and the last division a few u.
Codes, scales, paths and tokens are exact.
"""
import numpy as np
import pytest

import oracle
from oracle import speculative as sp
from weight_quantized_expert_b200 import api

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TOL_ROPE, TOL_TREE = 3e-6, 3e-5


def dev(a):
    import torch
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def ints(a):
    return None if a is None else dev(np.asarray(a, np.int32))


def f32(rng, *shape):
    return rng.standard_normal(shape).astype(np.float32)


# ---------------------------------------------------------------- rotation and norms

@pytest.mark.parametrize("T,hq,hk,rot,inter,norm", [
    (1, 10, 10, 128, False, False), (1, 10, 10, 128, True, True), (3, 20, 5, 64, False, True), (7, 1, 1, 34, False, True),
    (2, 3, 0, 2, True, False), (33, 128, 2, 96, True, True), (130, 11, 7, 126, False, False),
    (5, 3, 2, 96, False, True), (4, 2, 1, 8, False, False), (9, 40, 8, 120, False, True), (3, 2, 2, 2, False, True),
])
def test_rope(T, hq, hk, rot, inter, norm):
    rng = np.random.default_rng(T * 100 + hq)
    q, k = f32(rng, T, hq, 128), f32(rng, T, hk, 128) if hk else None
    gq = gk = None
    if norm:
        gq, gk = 1 + 0.3 * f32(rng, 128), None if hk == 2 else 1 + 0.3 * f32(rng, 128)
    pos = rng.integers(-5, 1_000_000, T)
    qo, ko = api.focr_qk_norm_rope(dev(q), dev(k), ints(pos), dev(gq), dev(gk), rot_dim=rot, interleaved=inter, norm=norm)
    for got, x, g in ((qo, q, gq), (ko, k, gk)):
        if x is not None:
            want = sp.qk_norm_rope(x, pos, g, rot=rot, interleaved=inter, norm=norm)
            assert np.abs(got.cpu().numpy() - want).max() <= TOL_ROPE * np.abs(want).max()


def test_rope_in_place_on_the_columns_of_a_fused_projection():
    import torch
    rng = np.random.default_rng(5)
    T, hq, hk = 5, 4, 2
    rows = f32(rng, T, (hq + 2 * hk) * 128)
    d = dev(rows)
    q, k = d[:, :hq * 128].view(T, hq, 128), d[:, hq * 128:(hq + hk) * 128].view(T, hk, 128)
    pos = np.arange(T) * 1000
    api.focr_qk_norm_rope(q, k, ints(pos), q_out=q, k_out=k)
    torch.cuda.synchronize()
    got = d.cpu().numpy()
    x = rows.reshape(T, -1, 128)
    want = sp.qk_norm_rope(x[:, :hq + hk], pos)
    assert np.abs(got.reshape(T, -1, 128)[:, :hq + hk] - want).max() <= TOL_ROPE * np.abs(want).max()
    np.testing.assert_array_equal(got[:, (hq + hk) * 128:], rows[:, (hq + hk) * 128:])   # the v columns are untouched


def test_rope_at_the_largest_positions():
    # theta^0 = 1: angle = pos; one turn is 2 pi, so the fp64 revolutions are off by pos / (2 pi) x 2^-52
    x = np.ones((2, 1, 128), np.float32)
    pos = np.array([2**31 - 1, -2**31])
    got = api.focr_qk_norm_rope(dev(x), None, ints(pos))[0].cpu().numpy()
    want = sp.qk_norm_rope(x, pos)
    assert np.abs(got - want).max() <= (TOL_ROPE + 2 * np.pi * 2**31 / 6.28 * 4 * 2.0**-52) * 1.5


def test_rope_of_zero_rows_with_norm():
    x = np.zeros((1, 2, 128), np.float32)
    got = api.focr_qk_norm_rope(dev(x), dev(x), ints([3]), norm=True)
    assert (got[0].cpu().numpy() == 0).all() and (got[1].cpu().numpy() == 0).all()


@pytest.mark.parametrize("inter,rot", [(True, 126), (True, 64), (True, 2), (False, 64)])
def test_rope_passes_infinities_behind_the_rotated_dims(inter, rot):
    x = f32(np.random.default_rng(rot), 2, 3, 128)
    x[:, :, 127], x[:, :, rot] = np.inf, -np.inf
    got = api.focr_qk_norm_rope(dev(x), None, ints([1, 70000]), rot_dim=rot, interleaved=inter)[0].cpu().numpy()
    np.testing.assert_array_equal(got[..., rot:], x[..., rot:])
    assert np.isfinite(got[..., :rot]).all()


# ---------------------------------------------------------------- cache writes and reads

def np_cache(rng, B, heads, cap, int4):
    out = []
    for _ in range(2):
        out += list(sp.quantise(f32(rng, B, heads, cap, 128), int4))
    return out


def dev_cache(c):
    return api.KVCache(*[dev(x) for x in c])


def check_write(rng, B, heads, cap, int4, rows, count, start, row0=None, index=None, n_max=None, wrap=False, scale=1.0):
    import torch
    k, v = f32(rng, rows, heads, 128) * np.float32(scale), f32(rng, rows, heads, 128)
    k[rows // 2] = 0.0                                    # a zero row
    k[0, 0, 3], k[0, 0, 64] = 127 * 0.5, 0.25             # ties: scale 1/2, quotient 1/2 -> 0
    c = np_cache(rng, B, heads, cap, int4)
    d = dev_cache(c)
    api.focr_kv_write(d, dev(k), dev(v), ints(count), ints(start), row0=ints(row0), index=ints(index), n_max=n_max, wrap=wrap)
    sp.kv_write(c, k, v, count, start, row0, index, n_max, wrap)
    torch.cuda.synchronize()
    for got, want in zip(d, c):
        np.testing.assert_array_equal(got.cpu().numpy(), want)
    return c, d


@pytest.mark.parametrize("int4", [False, True])
def test_prefill_write_of_ragged_sequences(int4):
    # flat rows with offsets; the third sequence is empty, the fourth does not fit, the fifth has a bad count
    check_write(np.random.default_rng(11), 6, 3, 40, int4, 120, [40, 7, 0, 30, 61, 1], [0, 33, 0, 11, 0, 39],
                row0=[0, 40, 47, 47, 77, 119], n_max=60)


@pytest.mark.parametrize("int4", [False, True])
def test_write_next_to_the_borders_of_the_rounding(int4):
    import torch
    # values at (k + 1/2) steps and one or two floats to either side, for steps of all mantissas
    rng = np.random.default_rng(29)
    top, rows = (7, 2000) if int4 else (127, 2000)
    m = (top * np.exp(rng.uniform(-20, 20, rows))).astype(np.float32)
    m[:4] = top, 2 * top, np.float32(1e-30), np.float32(1e30)
    step = m / np.float32(top)
    x = ((rng.integers(-top, top, (rows, 128)) + 0.5) * step[:, None].astype(np.float64)).astype(np.float32)
    for _ in range(2):
        x = np.where(rng.random(x.shape) < 0.4, np.nextafter(x, np.where(rng.random(x.shape) < 0.5, np.inf, -np.inf).astype(np.float32)), x)
    x = np.clip(x, -m[:, None], m[:, None])
    x[:, 5] = m
    c = api.new_kv_cache(1, 1, rows, api.W_INT4 if int4 else api.W_INT8)
    d = dev(x[:, None])
    api.focr_kv_write(c, d, d, ints([rows]), ints([0]))
    torch.cuda.synchronize()
    codes, scales = sp.quantise(x, int4)
    for got_c, got_s in ((c.k, c.k_scale), (c.v, c.v_scale)):
        np.testing.assert_array_equal(got_s.cpu().numpy()[0, 0], scales)
        np.testing.assert_array_equal(got_c.cpu().numpy()[0, 0], codes)


@pytest.mark.parametrize("int4", [False, True])
def test_ring_commit_by_path_with_wrap_and_more_tokens_than_slots(int4):
    rng = np.random.default_rng(12)
    index = np.stack([rng.permutation(150) for _ in range(4)])
    index[1, :3] = 9                                       # the same source row three times
    index[2, 1] = -1                                       # a source row before the first
    check_write(rng, 4, 2, 128, int4, 4 * 150, [5, 9, 150, 0], [126, 2**31 - 1, 1000, 7], index=index, n_max=150, wrap=True)


def test_write_leaves_out_rows_outside_the_source():
    check_write(np.random.default_rng(13), 2, 1, 16, False, 6, [4, 4], [0, 0], row0=[4, -2], n_max=4)


def test_write_of_tiny_and_huge_rows():
    for scale in (1e-44, 1e-38, 1e37):
        check_write(np.random.default_rng(14), 1, 2, 16, False, 8, [8], [3], n_max=8, scale=scale)
        check_write(np.random.default_rng(15), 1, 2, 16, True, 8, [8], [3], n_max=8, scale=scale)


def test_write_from_strided_columns_and_negative_start():
    import torch
    rng = np.random.default_rng(16)
    rows = f32(rng, 9, 6 * 128)
    d = dev(rows)
    k, v = d[:, 2 * 128:4 * 128].view(9, 2, 128), d[:, 4 * 128:].view(9, 2, 128)
    c = np_cache(rng, 1, 2, 20, False)
    g = dev_cache(c)
    api.focr_kv_write(g, k, v, ints([9]), ints([-1]), n_max=9)
    api.focr_kv_write(g, k, v, ints([9]), ints([11]), n_max=9)
    x = rows.reshape(9, 6, 128)
    sp.kv_write(c, x[:, 2:4], x[:, 4:], [9], [11], n_max=9)
    torch.cuda.synchronize()
    for got, want in zip(g, c):
        np.testing.assert_array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("heads,cap", [(1, 1), (3, 37), (10, 128)])
def test_read_back(int4, heads, cap):
    import torch
    rng = np.random.default_rng(17)
    B = 5
    c = np_cache(rng, B, heads, cap, int4)
    d = dev_cache(c)
    length = [0, cap, cap + 1, -1, (cap + 1) // 2]
    k, v = (torch.full((B, heads, cap, 128), 7.0, device="cuda") for _ in range(2))
    api.focr_kv_read(d, ints(length), k, v)
    for got, codes, scales in ((k, c[0], c[1]), (v, c[2], c[3])):
        want = np.full((B, heads, cap, 128), 7.0, np.float32)
        vals = sp.values(codes, scales).astype(np.float32)
        for b, n in enumerate(length):
            if 0 <= n <= cap:
                want[b, :, :n] = vals[b, :, :n]
        np.testing.assert_array_equal(got.cpu().numpy(), want)


# ---------------------------------------------------------------- tree attention

def random_tree(rng, N):
    return [int(rng.integers(max(-1, i - 5), i)) for i in range(N)]


MANY = 25000     # a capacity that even a small call splits into ranges


def wide_cache(cache, cap=MANY):
    """On the device with more rows, which hold scales that would show."""
    import torch
    out = []
    for x in dev_cache(cache):
        y = torch.full((*x.shape[:2], cap, *x.shape[3:]), float("nan") if x.ndim == 3 else 77, dtype=x.dtype, device="cuda")
        y[:, :, :x.shape[2]] = x
        out.append(y)
    return out


def check_tree(seed, B, N, hq, hk, Rcap, ref_len, n_gen, int4=False, parent="random", n_nodes=None, qscale=1.0, wide=None):
    import torch
    rng = np.random.default_rng(seed)
    q, k, v = f32(rng, B, N, hq, 128) * np.float32(qscale), f32(rng, B, N, hk, 128), f32(rng, B, N, hk, 128)
    ref, ring = np_cache(rng, B, hk, Rcap, int4), np_cache(rng, B, hk, 128, int4)
    # rows that no node may see hold what would show: NaN scales behind the reference block and in unused ring slots
    for b in range(B):
        for s in (ref[1], ref[3]):
            s[b, :, max(0, ref_len[b]):] = np.nan
        for s in (ring[1], ring[3]):
            s[b, :, max(0, n_gen[b]):] = np.nan
    if parent == "random":
        parent = [random_tree(rng, N) for _ in range(B)]
    if n_nodes is not None:
        for b in range(B):
            for x in (q, k, v):
                x[b, max(0, n_nodes[b]):] = np.nan
    out = torch.full((B, N, hq, 128), 7.0, device="cuda")
    dref = wide_cache(ref, wide) if wide else dev_cache(ref)
    assert bool(wide) == bool(api.focr_rswa_tree_workspace_bytes(B, N, hq, hk, dref[1].shape[2]))     # the kernel meant
    api.focr_rswa_tree(dev(q), dev(k), dev(v), dref, ints(ref_len), dev_cache(ring), ints(n_gen), ints(parent),
                       ints(n_nodes), out=out)
    ref, ring = (tuple(np.nan_to_num(sp.values(c[i], c[i + 1])) for i in (0, 2)) for c in (ref, ring))
    want = sp.rswa_tree(q, k, v, ref, ref_len, ring, n_gen, parent, n_nodes)
    got = out.cpu().numpy().astype(np.float64)
    for b in range(B):
        L = N if n_nodes is None else n_nodes[b]
        assert (got[b, L:] == 7.0).all()
        if L:
            vmax = max(np.abs(ref[1][b]).max(initial=0.0), np.abs(ring[1][b]).max(), np.abs(v[b, :L]).max())
            assert np.abs(got[b, :L] - want[b, :L]).max() <= TOL_TREE * max(1.0, qscale) * vmax, b
    return got


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("n", [0, 1, 5, 127, 128, 129, 600])
def test_single_token(n, int4):
    check_tree(100 + n, 1, 1, 10, 10, 289, [289], [n], int4, parent=None)


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("N,hq,hk", [(2, 10, 10), (3, 4, 2), (5, 2, 2), (8, 3, 3), (9, 2, 1), (16, 10, 10), (17, 1, 1),
                                     (33, 2, 2), (64, 2, 2), (16, 4, 1), (8, 16, 2), (1, 64, 1), (7, 8, 1)])
def test_trees_and_head_layouts(N, hq, hk, int4):
    check_tree(200 + N, 3, N, hq, hk, 75, [75, 0, 33], [600, 128, 40], int4)


@pytest.mark.parametrize("R", [0, 1, 15, 31, 32, 33, 63, 64, 65, 127, 255, 256, 257, 511, 513])
def test_reference_lengths_around_the_tiles(R):
    check_tree(300 + R, 2, 3, 2, 2, max(1, R), [R, R // 2], [R, 3])


def test_no_reference_and_nothing_generated():
    got = check_tree(31, 2, 4, 2, 2, 1, [0, 0], [0, 0], parent=[[-1, -1, -1, -1]] * 2)
    assert np.isfinite(got).all()      # each node sees itself alone


def test_chain_of_sixty_four_moves_the_window():
    check_tree(32, 2, 64, 2, 2, 10, [10, 3], [128, 70], parent=None)


def test_ragged_batch_with_empty_and_short_trees():
    check_tree(33, 5, 9, 10, 10, 300, [300, 0, 17, 299, 1], [1, 128, 500, 0, 129], n_nodes=[9, 0, 1, 8, 5])


@pytest.mark.parametrize("int4", [False, True])
def test_long_reference_block(int4):
    check_tree(34, 2, 5, 4, 2, 8192, [8191, 4100], [900, 40], int4)


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("N,hq,hk", [(1, 2, 2), (3, 4, 1), (16, 2, 2), (17, 1, 1), (16, 4, 2), (21, 2, 1), (33, 1, 1), (64, 1, 1), (16, 8, 2)])
def test_many_units_kernel_head_layouts(N, hq, hk, int4):
    # few units but a capacity that splits into ranges; lengths around its tiles of 128
    check_tree(400 + N, 3, N, hq, hk, 4300, [4300, 257, 128], [600, 127, 1], int4, wide=MANY)


@pytest.mark.parametrize("int4", [False, True])
def test_many_units_kernel_on_a_ragged_batch(int4):
    rng = np.random.default_rng(44)
    B = 170
    lens = [int(x) for x in rng.integers(0, 520, B)]
    lens[:8] = [0, 1, 127, 128, 129, 255, 256, 520]
    gen = [int(x) for x in rng.integers(0, 300, B)]
    gen[:4] = [0, 0, 1, 5]
    nodes = [int(x) for x in rng.integers(0, 4, B)]
    nodes[:4] = [3, 1, 0, 2]
    check_tree(45, B, 3, 2, 2, 520, lens, gen, int4, n_nodes=nodes, wide=1100)


def test_many_units_kernel_when_the_scores_keep_rising():
    import torch
    # keys ordered so that every tile has a new maximum: the bounds move all the time, and value scales grow too
    rng = np.random.default_rng(46)
    R, N = 4300, 4
    q = f32(rng, 1, N, 2, 128)
    k = f32(rng, 1, 2, R, 128) * 0.05 + q[:, 0][:, :, None] * np.linspace(0, 2, R, dtype=np.float32)[None, None, :, None]
    v = f32(rng, 1, 2, R, 128) * np.linspace(0.01, 3, R, dtype=np.float32)[None, None, :, None]
    for int4 in (False, True):
        ref = [x for y in (k, v) for x in sp.quantise(y, int4)]
        ring = np_cache(rng, 1, 2, 128, int4)
        kn, vn = f32(rng, 1, N, 2, 128), f32(rng, 1, N, 2, 128)
        got = api.focr_rswa_tree(dev(q), dev(kn), dev(vn), wide_cache(ref), ints([R]), dev_cache(ring), ints([40])).cpu().numpy()
        val = lambda c: (sp.values(c[0], c[1]), sp.values(c[2], c[3]))  # noqa: E731
        want = sp.rswa_tree(q, kn, vn, val(ref), [R], val(ring), [40])
        assert np.abs(got - want).max() <= TOL_TREE * np.abs(v).max()


def test_many_units_kernel_marks_invalid_sequences():
    import torch
    rng = np.random.default_rng(47)
    B, N, cap = 6, 3, 4300
    q, k = f32(rng, B, N, 2, 128), f32(rng, B, N, 2, 128)
    ref, ring = np_cache(rng, B, 2, cap, False), np_cache(rng, B, 2, 128, False)
    ref_len, n_gen, n_nodes = [MANY + 1, -1, 900, 4300, 4300, 1200], [5, 5, -1, 5, 5, 5], [3, 2, 3, 4, 3, 3]
    parent = [[-1, 0, 1]] * 4 + [[-1, 1, 0]] + [[-1, 0, -1]]
    out = torch.full((B, N, 2, 128), 7.0, device="cuda")
    api.focr_rswa_tree(dev(q), dev(k), dev(k), wide_cache(ref), ints(ref_len), dev_cache(ring), ints(n_gen), ints(parent),
                       ints(n_nodes), out=out)
    got = out.cpu().numpy()
    assert np.isnan(got[[0, 2, 3, 4]]).all() and np.isnan(got[1, :2]).all() and (got[1, 2] == 7.0).all()
    val = lambda c: (sp.values(c[0], c[1])[5:], sp.values(c[2], c[3])[5:])  # noqa: E731
    want = sp.rswa_tree(q[5:], k[5:], k[5:], val(ref), ref_len[5:], val(ring), n_gen[5:], parent[5:], n_nodes[5:])
    assert np.abs(got[5] - want[0]).max() <= TOL_TREE * 6


def test_many_sequences():
    check_tree(35, 70, 2, 2, 2, 40, [b % 41 for b in range(70)], [b * 7 for b in range(70)])


def test_large_scores_and_a_dominant_key():
    check_tree(36, 2, 6, 2, 2, 200, [200, 100], [300, 300], qscale=30.0)


def test_zero_queries_average_what_they_see():
    check_tree(37, 1, 6, 2, 2, 50, [50], [300], qscale=0.0)


def test_ring_positions_near_the_largest_int():
    check_tree(38, 2, 5, 2, 2, 8, [8, 2], [2**31 - 1, 2**31 - 3])


def test_invalid_sequences_get_nan_and_spare_the_others():
    import torch
    rng = np.random.default_rng(39)
    B, N = 6, 3
    q, k = f32(rng, B, N, 2, 128), f32(rng, B, N, 2, 128)
    ref, ring = np_cache(rng, B, 2, 16, False), np_cache(rng, B, 2, 128, False)
    ref_len, n_gen, n_nodes = [17, -1, 16, 16, 16, 16], [5, 5, -1, 5, 5, 5], [3, 2, 3, 4, 3, 3]
    parent = [[-1, 0, 1]] * 4 + [[-1, 1, 0]] + [[-1, 0, -1]]
    out = torch.full((B, N, 2, 128), 7.0, device="cuda")
    api.focr_rswa_tree(dev(q), dev(k), dev(k), dev_cache(ref), ints(ref_len), dev_cache(ring), ints(n_gen), ints(parent),
                       ints(n_nodes), out=out)
    got = out.cpu().numpy()
    assert np.isnan(got[[0, 2, 3, 4]]).all() and np.isnan(got[1, :2]).all() and (got[1, 2] == 7.0).all()
    assert np.isfinite(got[5]).all()


@pytest.mark.parametrize("cap", [300, MANY])      # one launch; ranges
@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("what", [np.nan, np.inf])
@pytest.mark.parametrize("which", [1, 3])         # key scales, value scales
def test_a_scale_that_is_no_number_reaches_those_who_see_it_alone(cap, int4, what, which):
    # a chain of three behind n = 200 tokens: token 72 is in the ring and seen by none, token 73 by the first node alone
    rng = np.random.default_rng(48)
    B, N, n = 3, 3, 200
    q, k, v = (f32(rng, B, N, 2, 128) for _ in range(3))
    ref, ring = np_cache(rng, B, 2, 300, int4), np_cache(rng, B, 2, 128, int4)
    ring[which][0, :, 72] = ring[which][1, :, 73] = ref[which][2, 0, 10] = what
    got = api.focr_rswa_tree(dev(q), dev(k), dev(v), wide_cache(ref, cap), ints([300] * B), dev_cache(ring), ints([n] * B)).cpu().numpy()
    ref[which][2, 0, 10] = 0
    ring[which][0, :, 72] = ring[which][1, :, 73] = 0
    val = lambda c: (sp.values(c[0], c[1]), sp.values(c[2], c[3]))  # noqa: E731
    want = sp.rswa_tree(q, k, v, val(ref), [300] * B, val(ring), [n] * B)
    ok = np.ones(got.shape, bool)
    ok[1, 0] = ok[2, :, 0] = False
    assert np.abs(got - want)[ok].max() <= TOL_TREE * max(np.abs(val(ref)[1]).max(), np.abs(val(ring)[1]).max(), np.abs(v).max())
    if which == 3 or np.isnan(what):      # (an infinite key's score may be that of a masked one)
        assert not np.isfinite(got[1, 0]).any() and not np.isfinite(got[2, :, 0]).any()


# ---------------------------------------------------------------- probabilities

@pytest.mark.parametrize("T,V,temp", [(1, 1, 1.0), (2, 5, 0.5), (3, 1023, 1.0), (1, 4096, 0.7), (5, 32001, 1.3),
                                      (2, 129280, 0.3), (1, 300007, 1.0), (150, 1000, 1.0), (3, 33333, 1.0), (5, 129281, 0.8),
                                      (150, 1001, 1.0), (40, 16382, 1.0), (40, 16385, 1.0), (2, 131071, 1.0), (7, 2, 1.0)])
def test_probs(T, V, temp):
    rng = np.random.default_rng(T + V)
    x = f32(rng, T, V) * 4
    if V > 4:
        x[0, 1] = -np.inf
    got = api.focr_token_probs(dev(x), temp).cpu().numpy().astype(np.float64)
    want = sp.token_probs(x, temp)
    span = np.where(np.isfinite(x), x.max(-1, keepdims=True) - x, 0.0) / temp
    assert (np.abs(got - want) <= (8 + 2 * span) * U * want + 1e-44).all()
    assert V <= 4 or got[0, 1] == 0.0


def test_probs_in_place_rows_without_a_finite_maximum_and_alignment():
    import torch
    rng = np.random.default_rng(41)
    x = f32(rng, 4, 777)
    x[1], x[2, 5], x[3, 6] = -np.inf, np.inf, np.nan
    d = dev(x)
    api.focr_token_probs(d, out=d)
    got = d.cpu().numpy()
    assert np.isnan(got[1:]).any(axis=1).all() and np.isnan(got[1]).all() and np.isnan(got[3]).all()
    np.testing.assert_allclose(got[0], sp.token_probs(x[:1])[0], rtol=3e-6)
    flat = torch.zeros(1 + 3 * 500, device="cuda")          # rows that start off a 16-byte boundary
    flat[1:] = dev(f32(rng, 1500))
    y = api.focr_token_probs(flat[1:].view(3, 500)).cpu().numpy()
    np.testing.assert_allclose(y, sp.token_probs(flat[1:].view(3, 500).cpu().numpy()), rtol=3e-6)
    for shift in (0, 1, 2, 3):                               # outputs aligned unlike the logits, and nothing beside them written
        out = torch.full((4 + 3 * 500,), 7.0, device="cuda")
        api.focr_token_probs(flat[1:].view(3, 500), out=out[shift:shift + 1500].view(3, 500))
        got = out.cpu().numpy()
        np.testing.assert_allclose(got[shift:shift + 1500].reshape(3, 500), y, rtol=1e-6)
        assert (got[:shift] == 7).all() and (got[shift + 1500:] == 7).all()


# ---------------------------------------------------------------- verification

def verify_case(rng, B, N, V, sharp=2.0, near=0.7):
    base = f32(rng, B, N + 1, V) * np.float32(sharp)
    target = sp.token_probs(base).astype(np.float32)
    draft = sp.token_probs((base + f32(rng, B, N + 1, V) * np.float32(near))[:, :N]).astype(np.float32)
    parent = np.array([random_tree(rng, N) for _ in range(B)])
    tokens = np.zeros((B, N), np.int32)
    for b in range(B):
        for i in range(N):
            p = draft[b, parent[b, i] + 1].astype(np.float64)
            tokens[b, i] = rng.choice(V, p=p / p.sum())
    return target, draft, tokens, parent, rng.random((B, N + 1), np.float32)


def check_verify(target, draft, tokens, parent, n_nodes, u):
    got = api.focr_spec_verify(dev(target), dev(draft), ints(tokens), ints(parent), ints(n_nodes), dev(u))
    want = sp.spec_verify(target, draft, tokens, parent, n_nodes, u)
    for g, w, name in zip(got, want, ("n_accept", "path", "next_token")):
        np.testing.assert_array_equal(g.cpu().numpy(), w, err_msg=name)
    return want


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("B,N,V", [(1, 1, 1), (3, 1, 2), (40, 4, 7), (20, 16, 100), (6, 64, 33), (5, 8, 1025), (2, 5, 20011),
                                   (1, 4, 129280), (3, 3, 300007)])
def test_verify(B, N, V, drawn):
    rng = np.random.default_rng(B * N + V)
    target, draft, tokens, parent, u = verify_case(rng, B, N, V)
    n_nodes = rng.integers(0, N + 1, B)
    n, _, _ = check_verify(target, draft if drawn else None, tokens, parent, n_nodes, u)
    check_verify(target, draft if drawn else None, tokens, parent if V % 2 else None, None, u)


def test_verify_rejects_siblings_down_to_the_residual():
    # many siblings of one root, a draft that knows little: most tests fail and the residual shrinks each time
    rng = np.random.default_rng(51)
    target, draft, _, _, u = verify_case(rng, 30, 12, 50, sharp=3.0, near=4.0)
    parent = np.full((30, 12), -1)
    tokens = np.stack([rng.choice(50, size=12, p=draft[b, 0].astype(np.float64) / draft[b, 0].astype(np.float64).sum()) for b in range(30)])
    n, _, _ = check_verify(target, draft, tokens, parent, None, np.minimum(u * 1.3, np.float32(0.999)))
    assert (n == 0).sum() >= 3
    check_verify(target, None, tokens, parent, None, u)      # chosen drafts, the same token twice among them


def test_verify_of_equal_distributions_and_of_one_hot_rows():
    rng = np.random.default_rng(52)
    target, _, tokens, parent, u = verify_case(rng, 8, 4, 64)
    n, _, _ = check_verify(target, target[:, :4].copy(), tokens, None, None, u)
    assert (n == 4).all()                                    # u q < p always holds for q = p and u < 1
    hot = np.zeros((8, 5, 64), np.float32)
    hot[:, :, 7] = 1.0
    draft = np.zeros((8, 4, 64), np.float32)
    draft[:, :, 7] = 1.0
    draft[:, :, 9] = 1.0                                     # not a distribution: the residual is empty after a rejection
    tok = np.where(np.arange(4) < 2, 7, 9) * np.ones((8, 1), int)
    n, _, nxt = check_verify(hot, draft, tok, None, None, u)
    assert (n == 2).all() and (nxt == 7).all()


def test_verify_samples_the_first_and_the_last_token():
    p = np.zeros((2, 2, 600), np.float32)
    p[:, :, [3, 599]] = 0.5
    u = np.array([[0.9, 0.0], [0.9, np.float32(1 - 2.0**-24)]], np.float32)
    _, _, nxt = check_verify(p, None, np.array([[5], [5]]), None, None, u)
    assert nxt.tolist() == [3, 599]


def test_verify_marks_invalid_sequences():
    rng = np.random.default_rng(53)
    target, draft, tokens, parent, u = verify_case(rng, 6, 4, 32)
    parent[:] = [-1, 0, 1, 2]
    n_nodes = [5, -1, 4, 4, 4, 2]
    tokens[2, 3], tokens[3, 0], parent[4, 2] = 32, -1, 2
    tokens[5, 3], parent[5, 3] = 99, 99                       # behind the last node: not looked at
    n, path, nxt = (x.cpu().numpy() for x in api.focr_spec_verify(dev(target), dev(draft), ints(tokens), ints(parent), ints(n_nodes), dev(u)))
    assert (n[:5] == -1).all() and (nxt[:5] == -1).all() and (path[:5] == -1).all()
    w = sp.spec_verify(target[5:], draft[5:], tokens[5:], parent[5:], n_nodes[5:], u[5:])
    assert n[5] == w[0][0] and nxt[5] == w[2][0]


# ---------------------------------------------------------------- streams, graphs and the whole step

def test_the_step_as_it_is_used_eager_on_another_stream_and_replayed():
    """rotate q and k -> write the prompt -> attend -> probabilities -> verify -> commit the path to the ring -> attend
    again, on a side stream, then captured into a graph and replayed on new inputs; and against the fp32 decode call."""
    import torch
    rng = np.random.default_rng(61)
    B, N, heads, R, V = 3, 6, 10, 100, 500
    hold = {}

    def fresh(seed):
        r = np.random.default_rng(seed)
        return dict(q=f32(r, B * N, heads, 128), k=f32(r, B * N, heads, 128), v=f32(r, B, N, heads, 128),
                    pk=f32(r, B * R, heads, 128), pv=f32(r, B * R, heads, 128), logits=3 * f32(r, B * (N + 1), V),
                    u=r.random((B, N + 1), np.float32), tokens=r.integers(0, V, (B, N)).astype(np.int32))

    a = fresh(1)
    d = {k: dev(x) for k, x in a.items()}
    pos, parent = ints(np.tile(400 + np.arange(N), B)), ints([[-1, 0, 0, 1, 2, 4]] * B)
    n_gen, ref_len, zero, full = ints([126, 0, 300]), ints([100, 50, 0]), ints([0] * B), ints([R] * B)

    def step(stream=None):
        ref, ring = api.new_kv_cache(B, heads, R), api.new_kv_cache(B, heads, 128)
        q, k = api.focr_qk_norm_rope(d["q"], d["k"], pos, norm=True, stream=stream)
        api.focr_kv_write(ref, d["pk"], d["pv"], full, zero, stream=stream)
        qt, kt = q.view(B, N, heads, 128), k.view(B, N, heads, 128)
        hold["out"] = api.focr_rswa_tree(qt, kt, d["v"], ref, ref_len, ring, zero, parent, stream=stream)
        p = api.focr_token_probs(d["logits"], 0.8, stream=stream).view(B, N + 1, V)
        n, path, nxt = api.focr_spec_verify(p, None, d["tokens"], parent, None, d["u"], stream=stream)
        api.focr_kv_write(ring, k, d["v"].view(B * N, heads, 128), n, n_gen, index=path, n_max=N, wrap=True, stream=stream)
        hold.update(ref=ref, ring=ring, q=q, k=k, probs=p, n=n, path=path, next=nxt)

    def check(a):
        g = {k: x.cpu().numpy() for k, x in hold.items() if k not in ("ref", "ring")}
        ps = pos.cpu().numpy()
        for x in ("q", "k"):
            assert np.abs(g[x] - sp.qk_norm_rope(a[x], ps, norm=True)).max() < 2e-5
        ref = [x.cpu().numpy() for x in hold["ref"]]
        want = [np.zeros_like(x) for x in ref]
        sp.kv_write(want, a["pk"], a["pv"], [R] * B, [0] * B, n_max=R)
        for x, y in zip(ref, want):
            np.testing.assert_array_equal(x, y)
        val = lambda c: (sp.values(c[0], c[1]), sp.values(c[2], c[3]))  # noqa: E731
        zr = (np.zeros((B, heads, 128, 128)),) * 2
        o = sp.rswa_tree(g["q"].reshape(B, N, heads, 128), g["k"].reshape(B, N, heads, 128), a["v"], val(ref), [100, 50, 0], zr,
                         [0] * B, parent.cpu().numpy())
        assert np.abs(g["out"] - o).max() <= TOL_TREE * 6
        n, path, nxt = sp.spec_verify(g["probs"], None, a["tokens"], parent.cpu().numpy(), None, a["u"])
        for x, y in (("n", n), ("path", path), ("next", nxt)):
            np.testing.assert_array_equal(g[x], y)
        ring = [np.zeros_like(x.cpu().numpy()) for x in hold["ring"]]
        sp.kv_write(ring, g["k"], a["v"].reshape(B * N, heads, 128), n, [126, 0, 300], index=path, n_max=N, wrap=True)
        for x, y in zip(hold["ring"], ring):
            np.testing.assert_array_equal(x.cpu().numpy(), y)

    step()
    check(a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    check(a)
    step(stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    check(a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (2, 3):
        b = fresh(seed)
        b["tokens"][:, 0] = sp.token_probs(b["logits"].reshape(B, N + 1, V)[:, 0]).argmax(-1)   # a draft worth accepting
        for k, x in b.items():
            d[k].copy_(torch.from_numpy(x))
        graph.replay()
        torch.cuda.synchronize()
        check(b)


def test_one_token_agrees_with_the_fp32_decode_attention():
    import torch
    rng = np.random.default_rng(62)
    B, R = 2, 289
    q, k, v = (f32(rng, B, 10, 128) for _ in range(3))
    ref, ring = dev_cache(np_cache(rng, B, 10, R, False)), dev_cache(np_cache(rng, B, 10, 128, False))
    rl, n = ints([289, 40]), [600, 60]
    kr, vr = api.focr_kv_read(ref, rl)
    kg, vg = api.focr_kv_read(ring, ints([128, 128]))
    got = api.focr_rswa_tree(dev(q)[:, None], dev(k)[:, None], dev(v)[:, None], ref, rl, ring, ints(n))
    want = api.focr_rswa_decode(dev(q), dev(k), dev(v), kr, vr, rl, kg, vg, ints([x + 1 for x in n]))
    torch.cuda.synchronize()
    assert (got[:, 0] - want).abs().max().item() <= 2 * TOL_TREE * 5


def test_same_inputs_give_the_same_bits():
    import torch
    rng = np.random.default_rng(63)
    c = dev_cache(np_cache(rng, 2, 2, 3000, False))
    ring = dev_cache(np_cache(rng, 2, 2, 128, False))
    q, k = dev(f32(rng, 2, 9, 4, 128)), dev(f32(rng, 2, 9, 2, 128))
    a, b = (api.focr_rswa_tree(q, k, k, c, ints([3000, 2000]), ring, ints([500, 9])) for _ in range(2))
    x = dev(f32(rng, 3, 50000))
    p1, p2 = api.focr_token_probs(x), api.focr_token_probs(x)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(p1, p2)


def test_two_calls_of_each_operator_at_once():
    import torch
    rng = np.random.default_rng(61)
    B, N, hk = 40, 3, 4

    def job():
        q, k, v = (dev(f32(rng, B, N, hk, 128)) for _ in range(3))
        ref = wide_cache(np_cache(rng, B, hk, 200, False), 1100)        # ranges: a workspace
        ring = dev_cache(np_cache(rng, B, hk, 128, False))
        target, draft, tokens, parent, u = verify_case(rng, B, N, 20001)
        return dict(q=q, k=k, v=v, ref=ref, ring=ring, n=ints(rng.integers(0, 300, B)), r=ints(rng.integers(0, 201, B)),
                    pos=ints(rng.integers(0, 9999, B * N)), logits=dev(f32(rng, 9, 20001)), target=dev(target), draft=dev(draft),
                    tokens=ints(tokens), parent=ints(parent), u=dev(u))

    def run(j, stream=None):
        s = dict(stream=stream)
        rot = api.focr_qk_norm_rope(j["q"].view(B * N, hk, 128), j["k"].view(B * N, hk, 128), j["pos"], norm=True, **s)
        out = api.focr_rswa_tree(j["q"], j["k"], j["v"], j["ref"], j["r"], j["ring"], j["n"], j["parent"], **s)
        p = api.focr_token_probs(j["logits"], 0.9, **s)
        ver = api.focr_spec_verify(j["target"], j["draft"], j["tokens"], j["parent"], None, j["u"], **s)
        return [*rot, out, p, *ver]

    jobs = [job() for _ in range(2)]
    alone = [run(j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(5):
        both = [run(j, s) for j, s in zip(jobs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(alone, both):
            for x, y in zip(a, b):
                assert torch.equal(x, y)
