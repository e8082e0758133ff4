"""Tree attention over caches whose scores climb from tile to tile: a block walks
16 steps of a unit and more (the other tests mostly give it one), so the softmax
references, in one kernel shared between rows, move again and again.

Tolerances: as in test_gpu_paged.py, and what fp32 scores of this size add. A
score is off by d = 2 D 2^-24 z + 2^-20 (1 + z), z = max_j scale sum |q k_j|, so
a probability moves by at most exp(2 d) - 1 relatively, and o by that times a =
sum_j p_j |v_j|.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import test_gpu_paged as T  # noqa: E402
from gpu_helpers import f64  # noqa: E402
from ranking_prefill_gb300 import lib  # noqa: E402

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
LN2 = 0.6931471805599453                 # as the scale: scores are then powers of two
ROWS, TILES = 2000, 16                   # cached rows of every request, their steps of 128

# query heads of the one kv head, D, nodes, least rows: 16, 32, 64 columns a tile, then
# one and two row tiles of the kernel for many rows
KINDS = [(2, 128, 1, 1), (4, 64, 3, 1), (4, 128, 8, 17), (2, 64, 13, 17), (4, 128, 16, 33), (3, 64, 20, 33),
         (4, 128, 20, 65), (4, 64, 33, 129), (2, 128, 100, 129)]


def batch(hq, D, n, low, blocks, seed=0, scale=LN2, lens=ROWS, ps=64):
    """Requests of n chained nodes over the same `lens` cached rows, as many as give
    each block `blocks` of them, one kv head. Components 0 to 3 of q and k are zero, the
    caller's; the others give scores of some units."""
    B = blocks * torch.cuda.get_device_properties(0).multi_processor_count
    t = T.Tree([lens], [n], hq, 1, D, ps, None, seed=seed, scale=scale, max_nodes=max(n, -(-low // hq)))
    t.lens, t.nodes = np.full(B, lens), np.full(B, n)
    t.cu = np.arange(B + 1) * n
    t.T = B * n
    t.table = np.repeat(t.table, B, 0)
    t.q = (T.randn(seed + 3, t.T, hq, D).float() * 0.125).to(BF16)
    t.k, t.v = T.randn(seed + 4, t.T, 1, D), T.randn(seed + 5, t.T, 1, D)
    for x in (t.q, t.k, t.kc):
        x[..., :4] = 0
    return t


def by_tile(t, c, values):
    """Component c of the cached keys: values[i] in tile i."""
    for i, x in enumerate(values):
        for j in range(i * 128, min((i + 1) * 128, int(t.lens[0])), t.ps):
            t.kc[int(t.table[0, j // t.ps]), :, 0, c] = float(x)


def check(t, requests, status=lib.MIS_OK):
    t.prepare()
    t.call()
    assert lib.mis_get_device_status(t.ws) == status
    got, gl = f64(t.o), f64(t.lse)
    o, ls, a, z = t.oracle(rows_of=requests)
    rows = np.concatenate([np.arange(t.cu[b], t.cu[b + 1]) for b in requests])
    d = 2.0 * t.D * 2.0 ** -24 * z + 2.0 ** -20 * (1 + z)
    tol = (2.0 ** -8 + 2.0 ** -12 + np.expm1(2 * d).T[:, :, None]) * a + 2.0 ** -8 * (1 + 2.0 ** -8) * np.abs(o)
    err = np.abs(got - o)[rows]
    assert (err <= tol[rows]).all(), (err - tol[rows]).max()
    e = np.abs(gl - ls)[:, rows]
    assert (e <= (d + 2.0 ** -20 * np.abs(ls))[:, rows]).all(), e.max()
    first = t.o.clone()
    t.o.fill_(5.0)
    t.call()
    torch.cuda.synchronize()
    assert torch.equal(first, t.o)
    return got, gl


def some(t):
    B = len(t.lens)
    return [0, 1, B // 2, B - 1]


@pytest.mark.parametrize("climb", [5.0, 8.5, 20.0, 30.0, 39.0, 60.0])
@pytest.mark.parametrize("hq,D,n,low", KINDS)
def test_one_head_climbs_while_the_others_stay(hq, D, n, low, climb):
    t = batch(hq, D, n, low, 2)
    by_tile(t, 0, range(TILES))
    t.q[:, 0, 0] = climb
    check(t, some(t))


@pytest.mark.parametrize("climb", [8.5, 30.0, 60.0])
@pytest.mark.parametrize("hq,D,n,low", KINDS)
@pytest.mark.parametrize("scale", [LN2, -LN2])
def test_climbing_and_falling_heads_in_units_cut_anywhere(hq, D, n, low, climb, scale):
    t = batch(hq, D, n, low, 2, seed=1, scale=scale)
    B = 2 * len(t.lens) // 3 + 1                        # pieces of units
    t.lens, t.nodes, t.cu, t.table = t.lens[:B], t.nodes[:B], t.cu[:B + 1], t.table[:B]
    t.T = B * n
    t.q, t.k, t.v = t.q[:t.T], t.k[:t.T], t.v[:t.T]
    by_tile(t, 0, range(TILES))
    for g, x in enumerate([climb, -climb, climb / 2, 0.0][:hq]):
        t.q[:, g, 0] = x
    check(t, some(t))


@pytest.mark.parametrize("hq,D,n,low", KINDS)
def test_heads_that_drift_apart_and_meet_again(hq, D, n, low):
    # the first head climbs alone, the second follows, then the first again, then the second
    t = batch(hq, D, n, low, 2, seed=2)
    t.q[:, 0, 0], t.q[:, 1, 1] = 30.0, 30.0
    by_tile(t, 0, [0, 1, 2, 3, 3, 3, 3, 3, 4, 5, 6, 6, 6, 6, 6, 6])
    by_tile(t, 1, [0, 0, 0, 0, 1, 2, 3, 3, 3, 3, 3, 4, 5, 6, 6, 6])
    check(t, some(t))


@pytest.mark.parametrize("hq,D,n,low", KINDS)
def test_nodes_climb_apart_too(hq, D, n, low):
    t = batch(hq, D, n, low, 2, seed=3)
    by_tile(t, 0, range(TILES))
    t.q[:, :, 0] = torch.linspace(-12, 40, t.T * hq, device="cuda").view(t.T, hq)[torch.randperm(t.T, device="cuda")]
    check(t, some(t))


@pytest.mark.parametrize("climb", [20.0, 39.0, 60.0])
@pytest.mark.parametrize("hq,D,n,low", KINDS)
def test_other_requests_climb(hq, D, n, low, climb):
    # rows of the requests that follow lie behind a request's own in its tile of Q
    t = batch(hq, D, n, low, 2, seed=4)
    by_tile(t, 0, range(TILES))
    t.q.view(len(t.lens), n, hq, D)[1::2, :, :, 0] = climb
    check(t, [0, 1, 2, len(t.lens) - 2])


@pytest.mark.parametrize("hq,D,n,low", KINDS)
def test_bits_do_not_depend_on_other_requests_queries(hq, D, n, low):
    t = batch(hq, D, n, low, 2, seed=5)
    by_tile(t, 0, range(TILES))
    t.prepare()
    t.call()
    q = t.q.view(len(t.lens), n, hq, D)
    mine = lambda: (t.o.view(len(t.lens), n, hq, D)[::2].clone(),  # noqa: E731
                    t.lse.view(hq, len(t.lens), n)[:, ::2].clone())
    want = mine()
    for x in (3.0, 20.0, 60.0, -60.0, float("inf"), float("nan")):
        q[1::2, :, :, 0] = x
        t.call()
        assert lib.mis_get_device_status(t.ws) == lib.MIS_OK
        for a, b in zip(mine(), want):
            assert torch.equal(a, b), x


# scores of any size: (scale, power) of a head whose products with the keys are whole
# numbers times 2^power, so exact in fp32
SIZES = [(1.0, 9), (1.0, 24), (1.0, 31), (-1.0, 33), (1.0, 100), (-1.0, 118), (1e20, 0), (1e20, 60), (-1e20, 30),
         (1e-20, 100)]


@pytest.mark.parametrize("scale,power", SIZES)
@pytest.mark.parametrize("down", [False, True])
@pytest.mark.parametrize("hq,D,n,low", KINDS)
def test_scores_of_any_size(hq, D, n, low, down, scale, power):
    # keys of one tile tie, so do two tiles; the other heads see every key alike.
    # Probabilities are 1 / m or 0, exactly, whatever the size
    t = batch(hq, D, n, low, 1, seed=6, scale=scale)
    for x in (t.q, t.k, t.kc):
        x.zero_()
    m = np.array([150, 100, 201, 7, 201, 200, 3, 9, 40, 201, 60, 61, 62, 63, 64, 1]) - (250 if down else 0)
    by_tile(t, 0, m * np.sign(scale))
    t.k[:, 0, 0] = (-255 if down else 0) * float(np.sign(scale))
    t.q[:, 0, 0] = 2.0 ** power
    t.prepare()
    t.call()
    assert lib.mis_get_device_status(t.ws) == lib.MIS_OK
    got, gl = f64(t.o), f64(t.lse)
    requests = some(t)
    rows = np.concatenate([np.arange(t.cu[b], t.cu[b + 1]) for b in requests])
    o, ls, a, _ = t.oracle(rows_of=requests)
    tol = (2.0 ** -8 + 2.0 ** -12) * a + 2.0 ** -8 * (1 + 2.0 ** -8) * np.abs(o)
    assert (np.abs(got - o)[rows] <= tol[rows]).all()
    with np.errstate(over="ignore"):
        want = ls[:, rows].astype(np.float32).astype(np.float64)        # past fp32's range: infinite
    inf = np.isinf(want)
    assert (gl[:, rows][inf] == want[inf]).all()
    e = np.abs(gl[:, rows] - np.where(inf, 0, want))[~inf]
    assert (e <= 2.0 ** -20 * (1 + np.abs(want[~inf]))).all(), e.max()


@pytest.mark.parametrize("lens", [[100, 110], [20000, 30000]])           # whole units mostly, and pieces
@pytest.mark.parametrize("where", ["node", "cache"])
@pytest.mark.parametrize("hq,D,n,low", KINDS)
def test_infinite_values_with_small_weights_reach_the_rows_that_see_them(hq, D, n, low, where, lens):
    # one cached row's scores lie 300 powers of two above all others
    nodes = [n, n]
    par = np.concatenate([[-1], np.arange(n - 1) // 2, [-1], np.arange(n - 1) // 2]).astype(int)
    t = T.Tree(lens, nodes, hq, 1, D, 64, par, seed=50, scale=LN2, max_nodes=max(n, -(-low // hq)))
    t.q.mul_(0.125)
    for x in (t.q, t.k, t.kc):
        x[..., 0] = 0
    t.q[..., 0] = 60.0
    t.kc[int(t.table[0, 1]), 7, 0, 0] = 5.0
    sees = np.zeros((2 * n, 2 * n), bool)
    for b in range(2):
        sees[b * n:b * n + n, b * n:b * n + n] = T.P.ancestors(par[b * n:b * n + n])
    want = [x.copy() for x in t.oracle()]
    if where == "node":
        j = min(1, n - 1)
        t.v[j, 0, 5], t.v[j, 0, 9] = float("inf"), float("nan")
        hit = sees[:, j]
    else:
        page = int(t.table[0, (lens[0] - 1) // 64])
        t.vc[page, 0, 0, 5], t.vc[page, 0, 0, 9] = float("inf"), float("nan")
        hit = np.arange(2 * n) < n
    t.prepare()
    t.call()
    assert lib.mis_get_device_status(t.ws) == lib.MIS_OK
    got = f64(t.o)
    if where == "node":
        assert (got[hit][:, :, 5] == np.inf).all()
    assert not np.isfinite(got[hit][:, :, 5]).any() and np.isnan(got[hit][:, :, 9]).all()
    for d in (5, 9):
        got[hit, :, d] = want[0][hit, :, d] = 0
    assert np.isfinite(got).all()
    d = 2.0 * D * 2.0 ** -24 * want[3] + 2.0 ** -20 * (1 + want[3])
    tol = (2.0 ** -8 + 2.0 ** -12 + np.expm1(2 * d).T[:, :, None]) * want[2] + \
        2.0 ** -8 * (1 + 2.0 ** -8) * np.abs(want[0])
    assert (np.abs(got - want[0]) <= tol).all()
