"""GPU parity of the operators over a state cache (drafted trees, ragged runs, copies) against the fp64
definitions, their reports of malformed indices, and a run of them together.

Tolerances.  A step of the recurrence in fp32 adds at most some 22 roundings of 2^-24 to an element, relative
to the largest term (16 in-thread and 3 shuffled additions of a dot product, the decay, the update), the map
of a step does not grow what came before by more than the terms' own size, and the longest runs here have 64
steps: 22 * 64 * 2^-24 = 8.4e-5 of the largest value, under the fp32 bar of 1e-4 that the other parity tests
use.  bf16 outputs add one rounding, 2^-8 of the value.  Where trees are taken on the tensor cores, a factor is two
bf16, 2^-17 off: for unit vectors of 128 channels a product of two is off by some 2^-16 / sqrt(128) = 1.3e-6, on a
path of 64 nodes by sqrt(64) times that, 1.1e-5.  Copies are exact."""
import numpy as np
import pytest

from oracle import operators as op
from tests.gpu_util import cuda_or_skip, f64

pytestmark = pytest.mark.gpu
BAR = 1e-4
HALF = {"bf16": 2.0 ** -8, "f32": 0.0}


def tokens(torch, seed, n, H, K, V, dtype, low=None):
    gen = torch.Generator().manual_seed(seed)
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    r = lambda d: torch.randn(n, H, d, generator=gen)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    alpha = torch.exp(-torch.nn.functional.softplus(r(K) + 1))
    if low is not None:
        alpha[torch.rand(alpha.shape, generator=gen) < 0.1] = low
    x = [unit(r(K)).to(td), unit(r(K)).to(td), r(V).to(td), alpha, torch.sigmoid(r(K)).to(td), torch.sigmoid(r(V)).to(td)]
    return [a.cuda() for a in x]


def make_pool(torch, seed, slots, H, K, V):
    return (0.2 * torch.randn(slots, H, K, V, generator=torch.Generator().manual_seed(seed))).cuda()


def i32(torch, v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def close(got, ref, dtype):
    got = f64(got)
    assert np.isfinite(got).all()
    bar = BAR * np.abs(ref).max() + HALF[dtype] * np.abs(ref)
    assert (np.abs(got - ref) <= bar).all(), f"worst {np.max(np.abs(got - ref) / bar):.2f} of the bar"


@pytest.fixture
def wait_limit():
    """Sets how often the bounded waits of this thread's calls poll; the usual limits again when the test ends."""
    import gated_delta_rule_96_b200 as g
    yield g.gdn2_set_wait_limit
    g.gdn2_set_wait_limit(-1)


def random_tree(rng, n, back):
    return [-1] + [int(rng.integers(max(-1, i - back), i)) for i in range(1, n)] if n else []


def run_tree(torch, g, x, pool, slots, sizes, parents, extra=0, most=None):
    total, H, V = x[0].shape[0], x[0].shape[1], x[2].shape[2]
    cu = np.concatenate([[0], np.cumsum(sizes)])
    assert cu[-1] + extra == total
    o = torch.full((total, H, V), float("nan"), dtype=x[0].dtype, device="cuda")
    ws = g.new_workspace(0)
    par = list(parents) + [-7] * extra
    before = pool.clone()
    g.gdn2_tree_fwd(*x, pool, i32(torch, slots), i32(torch, cu), i32(torch, par), o, most or max(list(sizes) + [0]),
                    workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(pool, before)
    ref = op.tree(*(f64(a) for a in x), f64(pool), slots, cu, par) if total - extra else None
    return o, ref, int(cu[-1]), g.gdn2_workspace_status(ws)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K,V", [(128, 128), (64, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("sizes", [[1], [2, 0, 5], [8, 3, 1, 0, 7], [17, 31, 32], [33, 64], [64, 63, 2, 48]])
def test_tree(dtype, K, V, sizes):
    torch, g = cuda_or_skip()
    rng, H = np.random.default_rng(sum(sizes)), 3
    x = tokens(torch, sum(sizes), sum(sizes) + 2, H, K, V, dtype)
    parents = sum((random_tree(rng, n, 9) for n in sizes), [])
    o, ref, rows, status = run_tree(torch, g, x, make_pool(torch, 1, 7, H, K, V), rng.permutation(7)[:len(sizes)].tolist(),
                                    sizes, parents, extra=2)
    assert status == 0
    close(o[:rows], ref[:rows], dtype)
    assert torch.isnan(o[rows:]).all()           # rows of no tree stay as they were


@pytest.mark.parametrize("seed", [0, 1, 2])
def test_tree_many_items(seed):
    """More (sequence, head) pairs than the GPU has SMs: trees of every size, empty and malformed ones between."""
    torch, g = cuda_or_skip()
    rng, H, B = np.random.default_rng(seed), 13, 48
    sizes = [int(n) for n in rng.choice([0, 1, 2, 7, 8, 9, 31, 32, 33, 40, 64], B)]
    cu, parents = np.concatenate([[0], np.cumsum(sizes)]), sum((random_tree(rng, n, 1 + 2 * (i % 8)) for i, n in enumerate(sizes)), [])
    x, pool, slots = tokens(torch, seed, cu[-1], H, 128, 128, "bf16"), make_pool(torch, seed, 60, H, 128, 128), rng.integers(-1, 60, B)
    ref = op.tree(*(f64(a) for a in x), f64(pool), slots, cu, parents)
    bad = [i for i in range(B) if sizes[i] and i % 7 == 3]
    for i in bad:
        parents[cu[i + 1] - 1] = sizes[i]
    o, ws = torch.full_like(x[2], float("nan")), g.new_workspace(0)
    g.gdn2_tree_fwd(*x, pool, i32(torch, slots), i32(torch, cu), i32(torch, parents), o, 64, workspace=ws)
    assert g.gdn2_workspace_status(ws) == (g.DEV_PARENT if bad else 0)
    left = sorted(r for i in bad for r in range(cu[i], cu[i + 1]))
    kept = sorted(set(range(cu[-1])) - set(left))
    assert torch.isnan(o[left]).all()
    close(o[kept], ref[kept], "bf16")


@pytest.mark.parametrize("items", [(1, 4), (8, 16)])
def test_tree_values_that_round_the_other_way(items):
    """What splitting the tensor cores' factors leaves of fp32 before o is rounded, on both kernels: an error of e of o's
    norm moves a value over a rounding border in proportion to e.  The couplings' split factors (2^-18 and 2^-18, rms a
    third of it, over 128 terms) would put o 4e-6 off and round one value in 240 the other way; with the largest, a node's
    own, in fp32 what is left is 2e-6, and the bar is one in 330.  fp32 is 1e-7 off: one in 10,000, bar 2,000."""
    torch, g = cuda_or_skip()
    batch, H = items
    n = 64 if batch > 1 else 32                   # 32 nodes of 4 items: CUDA cores
    x, pool = tokens(torch, 97, batch * n, H, 128, 128, "bf16"), make_pool(torch, 98, batch, H, 128, 128) / 2
    parents = sum((random_tree(np.random.default_rng(i), n, 12) for i in range(batch)), [])
    o, ref, _, status = run_tree(torch, g, x, pool, range(batch), [n] * batch, parents)
    assert status == 0
    other = (o.cpu() != torch.from_numpy(ref).bfloat16()).double().mean().item()
    assert other <= (1 / 330 if batch > 1 else 1 / 2000), 1 / other


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", ["chain", "star", "roots", "twos"])
@pytest.mark.parametrize("n", [6, 64])
def test_tree_shapes_on_a_zero_state_and_with_hard_decays(dtype, shape, n):
    torch, g = cuda_or_skip()
    parents = {"chain": [i - 1 for i in range(n)], "star": [-1] + [0] * (n - 1), "roots": [-1] * n,
               "twos": [-1] + [(i - 1) // 2 for i in range(1, n)]}[shape]
    for low in (None, 0.0, 1e-30):               # decays that end the past, or nearly
        x = tokens(torch, n, 2 * n, 2, 128, 128, dtype, low)
        if low is None:                          # and decays that keep it
            x[3].copy_(1 - 0.01 * x[3])
        o, ref, rows, status = run_tree(torch, g, x, make_pool(torch, 2, 3, 2, 128, 128), [-1, 2], [n, n], parents * 2)
        assert status == 0
        close(o, ref, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", [2.0 ** -20, 2.0 ** -39, 0.42, 0.3])
def test_tree_decays_whose_products_leave_the_range_along_a_path(dtype, decay):
    """The products pass 2^-80, and further down fp32's smallest number, on every long path, with short ones beside."""
    torch, g = cuda_or_skip()
    n = 64
    parents = [i - 1 for i in range(n)] + [-1] + [(i - 1) // 2 if i % 3 else i - 1 for i in range(1, n)]
    x = tokens(torch, 5, 2 * n, 3, 128, 128, dtype)
    x[3].fill_(decay)
    x[3][::5, :, 7] = 1.0                        # a channel that decays less than the others
    o, ref, rows, status = run_tree(torch, g, x, make_pool(torch, 6, 2, 3, 128, 128), [1, 0], [n, n], parents)
    assert status == 0
    close(o, ref, dtype)


@pytest.mark.parametrize("heads", [3, 5, 12, 25, 40])
def test_tree_sizes_of_every_kernel(heads):
    """The same trees as few and as many items, in calls for every most number of nodes: the kernels agree."""
    torch, g = cuda_or_skip()
    for n in (1, 5, 7, 8, 9, 10, 15, 16, 20, 21, 24, 40, 41):
        sizes = [n, max(1, n // 2), n, 0, n]
        parents = sum((random_tree(np.random.default_rng(n), m, 4) for m in sizes), [])
        x = tokens(torch, n, sum(sizes), heads, 128, 128, "bf16")
        o, ref, rows, status = run_tree(torch, g, x, make_pool(torch, n, 5, heads, 128, 128), [4, 2, -1, 1, 0], sizes, parents)
        assert status == 0
        close(o, ref, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [7, 40])
def test_tree_branches_do_not_touch_one_another(dtype, n):
    """NaN and infinities on one branch, and in another sequence's state, stay there."""
    torch, g = cuda_or_skip()
    parents = [-1, 0, 0] + [1 + (i % 2) for i in range(n - 3)]    # two branches below node 0
    x = tokens(torch, 3, 2 * n, 2, 128, 128, dtype)
    pool = make_pool(torch, 4, 3, 2, 128, 128)
    clean, ref, _, _ = run_tree(torch, g, x, pool, [0, 1], [n, n], parents * 2)
    sick = [i for i in range(n) if i == 1 or parents[i] == 1]
    y = [a.clone() for a in x]
    for a, bad in zip(y, (float("nan"), float("inf"), float("nan"), float("nan"), float("inf"), float("nan"))):
        a[sick] = bad
        a[n:] = bad                               # the whole second tree
    pool[1:] = float("nan")
    o = torch.empty_like(clean)
    g.gdn2_tree_fwd(*y, pool, i32(torch, [0, 1]), i32(torch, [0, n, 2 * n]), i32(torch, parents * 2), o, n)
    well = [i for i in range(n) if i not in sick]
    assert torch.equal(o[well], clean[well])
    assert not torch.isfinite(o[sick].float()).any()


@pytest.mark.parametrize("batch,n", [(20, 64), (3, 41)])
def test_tree_waits_that_run_out(wait_limit, batch, n):
    """Whichever wait of the tensor-core kernel runs out: the call ends and says so, a row of o is right or as it was,
    and the next call is as ever (no product is left on its way, no tensor memory held)."""
    torch, g = cuda_or_skip()
    H, sizes = 16, [n - i % 3 for i in range(batch)]
    cu = np.concatenate([[0], np.cumsum(sizes)])
    parents = sum((random_tree(np.random.default_rng(i), m, 1 + i) for i, m in enumerate(sizes)), [])
    x, pool = tokens(torch, n, cu[-1], H, 128, 128, "bf16"), make_pool(torch, n, batch, H, 128, 128)
    args = [i32(torch, a) for a in (range(batch), cu, parents)]
    want, ws = torch.full_like(x[2], float("nan")), g.new_workspace(0)
    g.gdn2_tree_fwd(*x, pool, *args, want, n, workspace=ws)
    assert g.gdn2_workspace_status(ws) == 0 and torch.isfinite(want).all()
    for polls in (0, 1, 2, 3, 4, 6, 8, 12, 16, 32, 64, 128, 256, 1024, 4096):
        o = torch.full_like(want, float("nan"))
        wait_limit(polls)
        g.gdn2_tree_fwd(*x, pool, *args, o, n, workspace=ws)
        wait_limit(-1)
        status = g.gdn2_workspace_status(ws, clear=True)
        assert status == g.DEV_WAIT or (status == 0 and torch.equal(o, want)), polls
        assert ((o == want).all(-1) | torch.isnan(o).all(-1)).all(), polls
        if polls == 0:
            assert status == g.DEV_WAIT and torch.isnan(o).all()
        g.gdn2_tree_fwd(*x, pool, *args, o, n, workspace=ws)
        assert g.gdn2_workspace_status(ws) == 0 and torch.equal(o, want), polls


def test_tree_reports_malformed_indices_and_serves_the_rest():
    torch, g = cuda_or_skip()
    H, n = 2, 5
    x = tokens(torch, 5, 6 * n, H, 128, 128, "f32")
    pool = make_pool(torch, 6, 4, H, 128, 128)
    good = [-1, 0, 1, 1, 0]
    base = dict(slots=[0, 1, 2, 3, 0, 1], cu=[n * i for i in range(7)], parents=good * 6)
    want = op.tree(*(f64(a) for a in x), f64(pool), base["slots"], base["cu"], base["parents"])

    def go(most=n, **change):
        c = {k: list(v) for k, v in base.items()}
        for key, (at, value) in change.items():
            c[key][at] = value
        o = torch.full((6 * n, H, 128), float("nan"), device="cuda")
        ws = g.new_workspace(0)
        g.gdn2_tree_fwd(*x, pool, i32(torch, c["slots"]), i32(torch, c["cu"]), i32(torch, c["parents"]), o, most, workspace=ws)
        return f64(o).reshape(6, n, H, 128), g.gdn2_workspace_status(ws)

    ref = want.reshape(6, n, H, 128)
    for change, bit, out in (({"slots": (2, 4)}, g.DEV_SLOT, [2]), ({"slots": (0, -2)}, g.DEV_SLOT, [0]),
                             ({"parents": (n + 2, 2)}, g.DEV_PARENT, [1]), ({"parents": (3 * n, -2)}, g.DEV_PARENT, [3]),
                             ({"parents": (4 * n + 1, 1 << 30)}, g.DEV_PARENT, [4]),
                             ({"cu": (6, 6 * n + 1)}, g.DEV_RANGE, [5]), ({"cu": (0, -1)}, g.DEV_RANGE, [0]),
                             ({"cu": (3, 2 * n - 1)}, g.DEV_RANGE, [2, 3])):
        o, status = go(**change)
        assert status == bit, (change, hex(status))
        for i in range(6):
            if i in out:
                assert np.isnan(o[i]).all(), (change, i)
            else:
                assert np.abs(o[i] - ref[i]).max() <= BAR * np.abs(ref).max()
    o, status = go(most=n - 1)
    assert status == g.DEV_RANGE and np.isnan(o).all()


def run_recurrent(torch, g, x, pool, src, dst, sizes, index=None, want_o=True, extra=0):
    H, V = x[0].shape[1], x[2].shape[2]
    cu = np.concatenate([[0], np.cumsum(sizes)])
    total = x[0].shape[0] if index is None else len(index)
    assert cu[-1] + extra == total
    o = torch.full((total, H, V), float("nan"), dtype=x[0].dtype, device="cuda") if want_o else None
    ws = g.new_workspace(0)
    ref = op.recurrent(*(f64(a) for a in x), f64(pool), src, dst, cu, index)
    g.gdn2_recurrent_fwd(*x, pool, i32(torch, src), i32(torch, dst), i32(torch, cu),
                         None if index is None else i32(torch, index), o, workspace=ws)
    torch.cuda.synchronize()
    assert g.gdn2_workspace_status(ws) == 0
    return o, ref[0], ref[1], int(cu[-1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K,V", [(128, 128), (64, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("H,sizes", [(1, [1]), (3, [1, 1, 1, 1]), (2, [2, 0, 9, 1]), (5, [8, 7, 17, 0, 3]), (16, [64]),
                                     (16, [1] * 20 + [5])])
def test_recurrent(dtype, K, V, H, sizes):
    torch, g = cuda_or_skip()
    rng, n = np.random.default_rng(len(sizes)), len(sizes)
    x = tokens(torch, sum(sizes) + H, sum(sizes) + 3, H, K, V, dtype)
    pool = make_pool(torch, 7, 2 * n + 1, H, K, V)
    slots = rng.permutation(2 * n + 1).tolist()
    for src, dst in ((slots[:n], slots[:n]), (slots[:n], slots[n:2 * n])):      # in place, and to other slots
        p = pool.clone()
        o, ref, after, rows = run_recurrent(torch, g, x, p, src, dst, sizes, extra=3)
        close(o[:rows], ref[:rows], dtype)
        close(p, after, "f32")
        assert torch.isnan(o[rows:]).all()
        idle = [s for s in range(2 * n + 1) if s not in dst]
        assert torch.equal(p[idle], pool[idle])


@pytest.mark.parametrize("K,V", [(128, 128), (64, 64)])
def test_recurrent_many_items(K, V):
    """More (sequence, head) pairs than the GPU has SMs, runs of every length between empty ones, a conflict."""
    torch, g = cuda_or_skip()
    rng, H, B = np.random.default_rng(K), 11, 60
    sizes = [int(n) for n in rng.choice([0, 1, 2, 3, 4, 5, 8, 21, 50], B)]
    cu, slots = np.concatenate([[0], np.cumsum(sizes)]), rng.permutation(2 * B + 1)
    src, dst = slots[:B].copy(), slots[B:2 * B].copy()
    src[3], dst[4], dst[10], src[11] = -1, -1, src[10], src[12]
    dst[20] = dst[21]
    x, pool = tokens(torch, K, cu[-1], H, K, V, "bf16"), make_pool(torch, K, 2 * B + 1, H, K, V)
    out = [20, 21]
    cu_ok = [i for i in range(B) if i not in out]
    ref, after = op.recurrent(*(f64(a) for a in x), f64(pool), src, [d if i not in out else -1 for i, d in enumerate(dst)], cu)
    o, ws = torch.full_like(x[2], float("nan")), g.new_workspace(0)
    g.gdn2_recurrent_fwd(*x, pool, i32(torch, src), i32(torch, dst), i32(torch, cu), None, o, workspace=ws)
    assert g.gdn2_workspace_status(ws) == g.DEV_CONFLICT
    kept = sorted(r for i in cu_ok for r in range(cu[i], cu[i + 1]))
    close(o[kept], ref[kept], "bf16")
    close(pool, after, "f32")
    assert torch.isnan(o[sorted(set(range(cu[-1])) - set(kept))]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_recurrent_gathers_clears_moves_and_only_reads(dtype):
    torch, g = cuda_or_skip()
    H, K, V = 4, 128, 128
    x = tokens(torch, 9, 12, H, K, V, dtype, low=0.0)
    pool = make_pool(torch, 8, 8, H, K, V)
    #        from zero, moved, cleared, not written, in place, neither read nor written
    src, dst = [-1, 3, -1, 0, 2, -1], [5, 6, 7, -1, 2, -1]
    sizes, index = [3, 0, 0, 4, 2, 1], [11, 0, 3, 3, 5, 5, 1, 2, 10, 4]
    p = pool.clone()
    o, ref, after, rows = run_recurrent(torch, g, x, p, src, dst, sizes, index)
    close(o, ref, dtype)
    close(p, after, "f32")
    assert torch.equal(p[6], pool[3]) and (p[7] == 0).all() and torch.equal(p[0], pool[0])
    q = pool.clone()
    run_recurrent(torch, g, x, q, src, dst, sizes, index, want_o=False)
    assert torch.equal(p, q)


def test_recurrent_is_the_decode_step_and_the_prefill():
    """Against the framework's own calls: runs of one against gdn2_decode_step, one run against gdn2_chunk_fwd
    on its fp32 path; the bars are those of the two calls' parity tests, once for each side."""
    torch, g = cuda_or_skip()
    B, H = 6, 3
    x = tokens(torch, 20, B, H, 128, 128, "bf16")
    pool = make_pool(torch, 21, B, H, 128, 128)
    S = pool.clone()
    o = g.recurrent_fwd(*x, pool, i32(torch, range(B)), i32(torch, range(B)), i32(torch, range(B + 1)))
    ref = g.decode_step(*x, S)
    close(o, f64(ref), "bf16")
    close(pool, f64(S), "f32")
    T = 64
    x = tokens(torch, 22, T, H, 64, 64, "f32")
    pool = make_pool(torch, 23, 1, H, 64, 64)
    ref_o, ref_S = g.chunk_fwd(*(a[None] for a in x), pool.clone())
    o = g.recurrent_fwd(*x, pool, i32(torch, [0]), i32(torch, [0]), i32(torch, [0, T]))
    assert np.abs(f64(o) - f64(ref_o)[0]).max() <= 2 * BAR * np.abs(f64(ref_o)).max()
    assert np.abs(f64(pool) - f64(ref_S)).max() <= 2 * BAR * np.abs(f64(ref_S)).max()


def test_recurrent_runs_of_any_length():
    """A run of 1.2 million tokens: the warps that wait for its end are not taken for stuck; its halves, one after the
    other, are the same blocks of four tokens."""
    torch, g = cuda_or_skip()
    n, half = 1200001, 600000
    gen = torch.Generator("cuda").manual_seed(1)
    r = lambda: torch.randn(n, 1, 64, generator=gen, device="cuda")  # noqa: E731
    x = [0.1 * r(), 0.1 * r(), r(), torch.sigmoid(r() + 2), torch.sigmoid(r()), torch.sigmoid(r())]
    pool = make_pool(torch, 1, 2, 1, 64, 64)
    pool[1] = pool[0]
    ws = g.new_workspace(0)
    o = g.recurrent_fwd(*x, pool, i32(torch, [0]), i32(torch, [0]), i32(torch, [0, n]), workspace=ws)
    first = g.recurrent_fwd(*(a[:half] for a in x), pool, i32(torch, [1]), i32(torch, [1]), i32(torch, [0, half]), workspace=ws)
    second = g.recurrent_fwd(*(a[half:] for a in x), pool, i32(torch, [1]), i32(torch, [1]), i32(torch, [0, n - half]), workspace=ws)
    assert g.gdn2_workspace_status(ws) == 0
    assert torch.equal(o[:half], first) and torch.equal(o[half:], second) and torch.equal(pool[0], pool[1])
    assert torch.isfinite(o).all() and o.abs().max() > 0


@pytest.mark.parametrize("B,slots", [(127, 400), (128, 400), (1000, 2600), (4100, 140000)])
def test_recurrent_conflicts_of_large_batches(B, slots):
    """Whatever finds them, and however many slots lie between: writers of one slot, writers of what another one reads, and
    updates in place whose slot another one reads are left out; shared sources, slots out of range, slots that differ by
    the size of a table, and sequences without a slot are no conflict."""
    torch, g = cuda_or_skip()
    rng = np.random.default_rng(B)
    p = rng.permutation(slots - 8)
    src, dst = p[:B].copy(), p[B:2 * B].copy()
    far = 1 << 17
    if slots > far + 8:
        at = np.flatnonzero(p[:2 * B] < slots - 8 - far)[:40]         # the same place, another slot
        both = np.concatenate([src, dst])
        for i, j in zip(at[::2], at[1::2]):
            if both[i] + far not in both:
                both[j] = both[i] + far
        src, dst = both[:B], both[B:]
    dst[0::9] = src[0::9]                                              # in place
    dst[1::9], src[2::9] = -1, -1
    src[3:12:9] = src[4]                                               # a source for several
    dst[22] = dst[23]                                                  # two writers
    dst[31] = src[33]                                                  # a writer of what 33 reads
    src[42] = dst[45]                                                  # 45 in place, read by 42
    dst[51] = src[51] = slots                                          # out of range, with the next line's reader
    src[52] = slots + 1
    dst[60] = src[61] = -1
    touch = {}
    for i in range(B):
        for s in {int(src[i]), int(dst[i])}:
            touch.setdefault(s, []).append(i)
    bad_slot = [i for i in range(B) if not (-1 <= src[i] < slots and -1 <= dst[i] < slots)]
    out = [i for i in range(B) if dst[i] >= 0 and i not in bad_slot and touch[int(dst[i])] != [i]]
    assert {22, 23, 31, 45} <= set(out)
    out += bad_slot
    x = tokens(torch, B, B, 1, 64, 64, "f32")
    pool = torch.randn(slots, 1, 64, 64, generator=torch.Generator("cuda").manual_seed(B), device="cuda")
    used = sorted({int(s) for s in np.concatenate([src, dst]) if 0 <= s < slots})
    row = {s: i for i, s in enumerate(used)}
    to_row = lambda a: [row.get(int(s), -1) for s in a]  # noqa: E731
    keep = pool[used].clone()
    kept_dst = dst.copy()
    kept_dst[out] = -1
    ref, after = op.recurrent(*(f64(a) for a in x), f64(keep), to_row(src), to_row(kept_dst), range(B + 1))
    o, ws = torch.full_like(x[2], float("nan")), g.new_workspace(0)
    total = pool.double().sum().item() - keep.double().sum().item()
    g.gdn2_recurrent_fwd(*x, pool, i32(torch, src.tolist()), i32(torch, dst.tolist()), i32(torch, range(B + 1)), None, o, workspace=ws)
    assert g.gdn2_workspace_status(ws) == g.DEV_CONFLICT | g.DEV_SLOT
    well = [i for i in range(B) if i not in set(out)]
    close(o[well], ref[well], "f32")
    assert torch.isnan(o[out]).all()
    close(pool[used], after, "f32")
    written = {row[int(s)] for s in kept_dst if s >= 0}
    idle = [i for i in range(len(used)) if i not in written]
    assert torch.equal(pool[used][idle], keep[idle])
    pool[used] = 0.0
    assert abs(pool.double().sum().item() - total) <= 1e-6 * max(1.0, abs(total))      # no other slot was touched


def test_recurrent_waits_for_long_runs_with_a_margin(wait_limit):
    """A poll a token, a quarter of what is added for a run's length, and nothing beside it, is enough for a long run."""
    torch, g = cuda_or_skip()
    n = 100000
    gen = torch.Generator("cuda").manual_seed(2)
    r = lambda: torch.randn(n, 1, 64, generator=gen, device="cuda")  # noqa: E731
    x = [0.1 * r(), 0.1 * r(), r(), torch.sigmoid(r() + 2), torch.sigmoid(r()), torch.sigmoid(r())]
    pool, ws = make_pool(torch, 1, 1, 1, 64, 64), g.new_workspace(0)
    wait_limit(n)
    o = g.recurrent_fwd(*x, pool, i32(torch, [0]), i32(torch, [0]), i32(torch, [0, n]), workspace=ws)
    assert g.gdn2_workspace_status(ws) == 0 and torch.isfinite(o).all()


def test_recurrent_reports_malformed_indices_and_conflicts():
    torch, g = cuda_or_skip()
    H, n = 2, 3
    x = tokens(torch, 10, 12, H, 64, 128, "f32")
    pool = make_pool(torch, 11, 8, H, 64, 128)
    base = dict(src=[0, 1, 2, -1], dst=[0, 4, 5, 6], cu=[0, 3, 6, 9, 12], index=list(range(12)))
    ref, after = op.recurrent(*(f64(a) for a in x), f64(pool), *(base[k] for k in ("src", "dst", "cu", "index")))
    cases = (({"src": (1, 8)}, g.DEV_SLOT, [1]), ({"dst": (2, -2)}, g.DEV_SLOT, [2]), ({"dst": (3, 99)}, g.DEV_SLOT, [3]),
             ({"index": (4, 12)}, g.DEV_INDEX, [1]), ({"index": (9, -1)}, g.DEV_INDEX, [3]),
             ({"cu": (4, 13)}, g.DEV_RANGE, [3]), ({"cu": (0, -3)}, g.DEV_RANGE, [0]),
             ({"dst": (1, 5)}, g.DEV_CONFLICT, [1, 2]),          # two writers of one slot: neither writes
             ({"dst": (3, 2)}, g.DEV_CONFLICT, [3]),             # a writer of a slot that another one reads
             ({"src": (2, 0)}, g.DEV_CONFLICT, [0]))             # the same, seen from an update in place
    for change, bit, out in cases:
        c = {k: list(v) for k, v in base.items()}
        for key, (at, value) in change.items():
            c[key][at] = value
        p, ws = pool.clone(), g.new_workspace(0)
        o = torch.full((12, H, 128), float("nan"), device="cuda")
        g.gdn2_recurrent_fwd(*x, p, i32(torch, c["src"]), i32(torch, c["dst"]), i32(torch, c["cu"]), i32(torch, c["index"]), o,
                             workspace=ws)
        assert g.gdn2_workspace_status(ws) == bit, change
        for i in range(4):
            rows = o[3 * i:3 * i + 3]
            if i in out:
                assert torch.isnan(rows).all(), (change, i)
            elif not ("src" in change and change["src"][0] == i):
                assert np.abs(f64(rows) - ref[3 * i:3 * i + 3]).max() <= BAR * np.abs(ref).max(), (change, i)
        written = {c["dst"][i] for i in range(4) if i not in out}
        idle = [s for s in range(8) if s not in written]
        assert torch.equal(p[idle], pool[idle]), change


@pytest.mark.parametrize("H,sizes", [(16, [40, 0, 300, 1, 7, 3, 90, 12, 1, 5, 2, 33]),    # a CTA holds a head's columns
                                     (2, [700, 0, 2])])                                  # they are split over CTAs
def test_recurrent_waits_that_run_out(wait_limit, H, sizes):
    """Whichever wait runs out: the call ends and says so, and a column of a state is either its run's last one or as it
    was.  Reported once, the next call is as ever."""
    torch, g = cuda_or_skip()
    n = len(sizes)
    x, pool = tokens(torch, H, sum(sizes), H, 128, 128, "bf16"), make_pool(torch, H, 2 * n, H, 128, 128)
    src = list(range(n - 1)) + [-1]
    for dst in (list(range(n)), list(range(n, 2 * n))):                  # in place, and to other slots
        args = [i32(torch, a) for a in (src, dst, np.concatenate([[0], np.cumsum(sizes)]))]
        want, ws = pool.clone(), g.new_workspace(0)
        o_want = torch.full_like(x[2], float("nan"))
        g.gdn2_recurrent_fwd(*x, want, *args, None, o_want, workspace=ws)
        assert g.gdn2_workspace_status(ws) == 0
        for polls in (0, 1, 2, 3, 4, 6, 8, 12, 16, 32, 64, 256, 4096):
            p, o = pool.clone(), torch.full_like(x[2], float("nan"))
            wait_limit(polls)
            g.gdn2_recurrent_fwd(*x, p, *args, None, o, workspace=ws)
            wait_limit(-1)
            status = g.gdn2_workspace_status(ws, clear=True)
            new, old = (p == want).all(-2), (p == pool).all(-2)          # by slot, head and column
            assert (new | old).all(), polls
            if n > 10:                                                   # a head's columns go together
                assert (new.all(-1) | old.all(-1)).all(), polls
            if status == 0:
                assert torch.equal(p, want) and torch.equal(o, o_want), polls
            else:
                assert status == g.DEV_WAIT
            if polls == 0:
                assert status == g.DEV_WAIT and old.all() and torch.isnan(o).all()
        g.gdn2_recurrent_fwd(*x, pool, *args, None, o, workspace=ws)
        assert g.gdn2_workspace_status(ws) == 0 and torch.equal(pool, want) and torch.equal(o, o_want)


@pytest.mark.parametrize("slots,shape,n", [(5, (1, 64, 64), 1), (9, (3, 64, 128), 4), (40, (2, 128, 128), 33),
                                           (300, (1, 64, 64), 250), (1100, (1, 4), 1024), (2000, (3, 64, 64), 1024)])
def test_state_copy(slots, shape, n):
    torch, g = cuda_or_skip()
    rng = np.random.default_rng(n)
    pool = torch.randn(slots, *shape, generator=torch.Generator().manual_seed(n)).cuda()
    perm = rng.permutation(slots)
    cyc = perm[:n]
    cases = [("reorder in place", cyc, np.roll(cyc, 1)), ("fork", perm[:n], np.full(n, perm[-1])),
             ("random, with repeats", rng.integers(-1, slots, n), rng.integers(-1, slots, n)),
             ("clear", perm[:n], np.full(n, -1)), ("one destination", np.full(n, 2), rng.integers(0, slots, n))]
    for name, dst, src in cases:
        p, ws = pool.clone(), g.new_workspace(0)
        g.gdn2_state_copy(p, p, i32(torch, dst), i32(torch, src), workspace=ws)
        assert np.array_equal(p.cpu().numpy(), op.state_copy(pool.cpu().numpy(), pool.cpu().numpy(), dst, src)), name
        assert g.gdn2_workspace_status(ws) == 0
    other = torch.randn(slots + 3, *shape, device="cuda")
    keep, dst, src = other.clone(), rng.permutation(slots + 3)[:n], rng.integers(0, slots, n)
    g.gdn2_state_copy(other, pool, i32(torch, dst), i32(torch, src))
    assert np.array_equal(other.cpu().numpy(), op.state_copy(keep.cpu().numpy(), pool.cpu().numpy(), dst, src))


@pytest.mark.parametrize("slots,shape,n", [(5, (2, 64, 64), 4), (300, (4, 128, 128), 250)])
def test_state_copy_waits_that_run_out(wait_limit, slots, shape, n):
    """Whichever wait runs out: the call ends and says so, and every value is the source's or as it was."""
    torch, g = cuda_or_skip()
    pool = torch.randn(slots, *shape, generator=torch.Generator().manual_seed(n)).cuda()
    order = np.random.default_rng(n).permutation(slots)
    for dst, src in ((order[:n], np.roll(order[:n], 1)), (order[:n // 2], order[n // 2:n // 2 * 2])):  # a reorder, a copy
        to, frm, ws = i32(torch, dst), i32(torch, src), g.new_workspace(0)
        want = pool.clone()
        g.gdn2_state_copy(want, want, to, frm, workspace=ws)
        assert g.gdn2_workspace_status(ws) == 0 and torch.equal(want[dst], pool[src])
        for polls in (0, 1, 2, 3, 4, 8, 16, 64, 1024):
            p = pool.clone()
            wait_limit(polls)
            g.gdn2_state_copy(p, p, to, frm, workspace=ws)
            wait_limit(-1)
            status = g.gdn2_workspace_status(ws, clear=True)
            assert ((p == want) | (p == pool)).all(), polls
            if status == 0:
                assert torch.equal(p, want), polls
            else:
                assert status == g.DEV_WAIT
            if polls == 0:
                assert status == g.DEV_WAIT and torch.equal(p, pool)
        g.gdn2_state_copy(pool, pool, to, frm, workspace=ws)
        assert g.gdn2_workspace_status(ws) == 0 and torch.equal(pool, want)


def test_state_copy_reports_bad_slots_and_serves_the_rest():
    torch, g = cuda_or_skip()
    pool = make_pool(torch, 12, 6, 1, 64, 64)
    p, ws = pool.clone(), g.new_workspace(0)
    g.gdn2_state_copy(p, p, i32(torch, [0, 6, 1, 2, -2]), i32(torch, [3, 0, 6, 4, 5]), workspace=ws)
    assert g.gdn2_workspace_status(ws, clear=True) == g.DEV_SLOT and g.gdn2_workspace_status(ws) == 0
    want = pool.clone()
    want[0], want[2] = pool[3], pool[4]
    assert torch.equal(p, want)


def test_one_layer_of_a_larger_pool():
    """Every call on one layer's part of a pool of all layers: the other layers stay as they were."""
    torch, g = cuda_or_skip()
    whole = make_pool(torch, 13, 6 * 3, 2, 128, 64).view(6, 3, 2, 128, 64)
    keep, layer = whole.clone(), whole[:, 1]
    x = tokens(torch, 14, 5, 2, 128, 64, "f32")
    par, cu, slots = [-1, 0, 0, 2, 1], [0, 5], [4]
    o = g.tree_fwd(*x, layer, i32(torch, slots), i32(torch, cu), i32(torch, par), 5)
    close(o, op.tree(*(f64(a) for a in x), f64(layer), slots, cu, par), "f32")
    ref, after = op.recurrent(*(f64(a) for a in x), f64(layer), slots, [2], cu)
    o = g.recurrent_fwd(*x, layer, i32(torch, slots), i32(torch, [2]), i32(torch, cu))
    close(o, ref, "f32")
    close(layer, after, "f32")
    now = layer.clone()
    g.gdn2_state_copy(layer, layer, i32(torch, [0, 5]), i32(torch, [5, 0]))
    assert torch.equal(layer[0], now[5]) and torch.equal(layer[5], now[0])
    assert torch.equal(whole[:, [0, 2]], keep[:, [0, 2]])


def test_copies_with_the_first_slot_of_a_layer_alone():
    """One slot of a strided cache, a part of that cache: to it, and from it, with a clear among the copies."""
    torch, g = cuda_or_skip()
    whole = make_pool(torch, 17, 6 * 3, 2, 64, 64).view(6, 3, 2, 64, 64)
    keep, layer = whole.clone(), whole[:, 1]
    now = layer.clone()
    g.gdn2_state_copy(layer[:1], layer, i32(torch, [0]), i32(torch, [3]))
    assert torch.equal(layer[0], now[3]) and torch.equal(layer[1:], now[1:])
    g.gdn2_state_copy(layer, layer[:1], i32(torch, [4, 0, 2]), i32(torch, [0, -1, 0]))
    assert torch.equal(layer[4], now[3]) and torch.equal(layer[2], now[3]) and not layer[0].any()
    assert torch.equal(layer[[1, 3, 5]], now[[1, 3, 5]])
    assert torch.equal(whole[:, [0, 2]], keep[:, [0, 2]])


def test_offsets_past_32_bits():
    """The last slots of a cache of more than 2^32 floats."""
    torch, g = cuda_or_skip()
    H, slots = 16, 16500                      # 262,144 floats a slot: 4.3e9 in all, 17 GB
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free device memory")
    pool = torch.zeros(slots, H, 128, 128, device="cuda")
    last, first = slots - 1, slots - 2
    pool[last] = make_pool(torch, 15, 1, H, 128, 128)[0]
    x = tokens(torch, 16, 3, H, 128, 128, "bf16")
    small = pool[last:].clone()
    o = g.tree_fwd(*x, pool, i32(torch, [last]), i32(torch, [0, 3]), i32(torch, [-1, 0, 0]), 3)
    close(o, op.tree(*(f64(a) for a in x), f64(small), [0], [0, 3], [-1, 0, 0]), "bf16")
    o = g.recurrent_fwd(*x, pool, i32(torch, [last]), i32(torch, [first]), i32(torch, [0, 3]))
    ref, after = op.recurrent(*(f64(a) for a in x), f64(small), [0], [0], [0, 3])
    close(o, ref, "bf16")
    close(pool[first], after[0], "f32")
    g.gdn2_state_copy(pool, pool, i32(torch, [first - 1]), i32(torch, [first]))
    assert torch.equal(pool[first - 1], pool[first]) and not pool[:first - 1].any()


def test_calls_on_a_side_stream_allocate_there():
    """`stream=` without a workspace: the outputs and the workspace are the stream's, while the current stream is
    kept busy."""
    torch, g = cuda_or_skip()
    H = 3
    x = tokens(torch, 50, 6, H, 128, 128, "bf16")
    pool = make_pool(torch, 51, 4, H, 128, 128)
    par, cu, slots = [-1, 0, 0, 1, -1, 0], [0, 4, 6], [1, 2]
    want_tree = g.tree_fwd(*x, pool, i32(torch, slots), i32(torch, cu), i32(torch, par), 4)
    p = pool.clone()
    want_rec = g.recurrent_fwd(*x, p, i32(torch, slots), i32(torch, [3, 0]), i32(torch, cu))
    idx = i32(torch, slots), i32(torch, cu), i32(torch, par), i32(torch, [3, 0])
    o, gate, w = x[2].reshape(-1, 128), x[5].reshape(-1, 128), torch.ones(128, device="cuda")
    want_norm = g.gated_norm_bwd(o, gate, w, gate)
    side, busy = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for _ in range(3):
        for _ in range(4):
            busy = busy @ busy * 1e-2                   # the current stream lags behind
        a = g.tree_fwd(*x, pool, idx[0], idx[1], idx[2], 4, stream=side)
        b = g.recurrent_fwd(*x, pool, idx[0], idx[3], idx[1], stream=side)
        c = g.gated_norm_bwd(o, gate, w, gate, stream=side)
        side.synchronize()
        with torch.cuda.stream(side):
            assert torch.equal(a, want_tree) and torch.equal(b, want_rec) and torch.equal(pool, p)
            assert all(torch.equal(s, t) for s, t in zip(c, want_norm))
        side.synchronize()
    torch.cuda.synchronize()


def test_malformed_indices_without_a_workspace_are_reported():
    """Calls that are given no workspace report to the device's shared status, on any stream and from a graph, with no
    allocation of their own."""
    torch, g = cuda_or_skip()
    x, pool = tokens(torch, 72, 6, 2, 64, 64, "bf16"), make_pool(torch, 73, 4, 2, 64, 64)
    good, bad, out, cu = i32(torch, [0, 1]), i32(torch, [0, 4]), i32(torch, [2, 3]), i32(torch, [0, 3, 6])
    par, wrong, src = i32(torch, [-1, 0, 0] * 2), i32(torch, [-1, 0, 0, -1, 1, 0]), i32(torch, [1, 1])
    keep, o = pool.clone(), torch.full_like(x[2], float("nan"))
    g.gdn2_state_copy(pool, pool, out, good)                       # the shared workspace is there from here on
    g.gdn2_shared_status()
    assert torch.equal(pool[2:], keep[:2])
    calls = [(lambda st: g.gdn2_tree_fwd(*x, pool, good, cu, wrong, o, 3, stream=st), g.DEV_PARENT),
             (lambda st: g.gdn2_tree_fwd(*x, pool, bad, cu, par, o, 3, stream=st), g.DEV_SLOT),
             (lambda st: g.gdn2_recurrent_fwd(*x, pool, good, bad, cu, None, None, stream=st), g.DEV_SLOT),
             (lambda st: g.gdn2_state_copy(pool, pool, out, bad, stream=st), g.DEV_SLOT),
             (lambda st: g.gdn2_state_copy(pool, pool, out, src, stream=st), 0)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for call, bits in calls:
        for st in (None, side):
            before = torch.cuda.memory_stats()["allocation.all.allocated"]
            call(st)
            made = torch.cuda.memory_stats()["allocation.all.allocated"] - before
            side.synchronize()
            assert g.gdn2_shared_status(clear=False) == bits and g.gdn2_shared_status("cuda:0") == bits
            assert g.gdn2_shared_status() == 0 and made == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.tree_fwd(*x, pool, bad, cu, par, 3)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert g.gdn2_shared_status() == g.DEV_SLOT and g.gdn2_shared_status() == 0


def test_a_call_captured_before_any_other():
    """The first call of a process, captured, without a workspace: the graph's own."""
    torch, g = cuda_or_skip()
    x, pool = tokens(torch, 74, 3, 2, 64, 64, "bf16"), make_pool(torch, 75, 2, 2, 64, 64)
    args = i32(torch, [1]), i32(torch, [0, 3]), i32(torch, [-1, 0, 1])
    want, kept = g.tree_fwd(*x, pool, *args, 3), dict(g._shared)
    try:
        g._shared.clear()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o = g.tree_fwd(*x, pool, *args, 3)
        assert not g._shared
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want)
    finally:
        g._shared.update(kept)


def test_calls_behind_one_another_see_what_the_last_one_wrote():
    """Chains of calls with nothing between them, each of which reads what the one before wrote (a launch is prepared
    while that one still runs), against the same calls one at a time; eager and in a graph."""
    torch, g = cuda_or_skip()
    x = tokens(torch, 3, 12, 16, 128, 128, "bf16")
    weight = torch.ones(2048, device="cuda")
    slots, cu, parents = i32(torch, [0, 1, 2]), i32(torch, [0, 4, 8, 12]), i32(torch, [-1, 0, 1, 1] * 3)
    to, frm = i32(torch, [1, 2, 3, 0]), i32(torch, [0, 1, 2, 3])
    ws, first = g.new_workspace(0), make_pool(torch, 3, 4, 16, 128, 128)

    def chain(pool, o, rows, between):
        for _ in range(12):
            g.gdn2_recurrent_fwd(*x, pool, slots, slots, cu, None, o, workspace=ws)
            between()
            g.gdn2_state_copy(pool, pool, to, frm, workspace=ws)
            between()
            g.gdn2_tree_fwd(*x, pool, slots, cu, parents, o, 4, workspace=ws)
            between()
            g.gdn2_add_norm_fwd(o.view(12, 2048), rows, None, weight, rows, o.view(12, 2048))
            between()
            g.gdn2_gated_norm_fwd(o, x[2], weight[:128], x[2])
            between()
            pool.mul_(0.99)
            between()
            g.decode_step(*(a[:4].contiguous() for a in x), pool)

    def run(between, graph=None):
        pool, o, rows, v = first.clone(), torch.zeros_like(x[2]), torch.zeros(12, 2048, device="cuda").bfloat16(), x[2].clone()
        torch.cuda.synchronize()
        if graph is None:
            chain(pool, o, rows, between)
        else:
            with torch.cuda.graph(graph):
                chain(pool, o, rows, between)
            graph.replay()
        torch.cuda.synchronize()
        out = [pool, o, rows, x[2].clone()]
        x[2].copy_(v)
        return out
    want = run(torch.cuda.synchronize)
    assert all(torch.isfinite(a.float()).all() for a in want)
    for got in [run(lambda: None) for _ in range(5)] + [run(lambda: None, torch.cuda.CUDAGraph())]:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert g.gdn2_workspace_status(ws) == 0


def test_every_input_may_be_what_the_kernel_before_wrote():
    """Tokens, weights, slots, counts, parents and indices, all of them written by the call right before (a copy of a large
    slot that ends with them), with nothing between: each call reads this turn's, not the turn's before."""
    torch, g = cuda_or_skip()
    floats = 1 << 24
    pool = torch.zeros(3, floats, device="cuda")                   # two turns' inputs, and where the calls read them
    at = [floats]

    def place(*pair):
        """Two turns' values of one input, at the slots' end; the input itself."""
        first, size = pair[0], pair[0].numel()
        at[0] -= -(-size * first.element_size() // 16) * 4
        views = [pool[i, at[0]:].view(first.dtype)[:size].view(first.shape) for i in range(3)]
        for view, value in zip(views, pair):
            view.copy_(value)
        return views[2]

    ints = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    H, n = 3, 44
    args = {}
    for few in (12, n):                                            # trees of both kernels
        turns = [tokens(torch, 80 + few + i, few, H, 128, 128, "bf16") for i in range(2)]
        trees = [ints(*random_tree(np.random.default_rng(i), few - 4, 6), -1, 0, 0, 1) for i in range(2)]
        args[few] = dict(x=[place(a, b) for a, b in zip(*turns)], parents=place(*trees),
                         cu=place(ints(0, few - 4, few), ints(0, few - 4, few - 1)), slots=place(ints(0, 1), ints(1, 0)),
                         index=place(*(torch.randperm(few, generator=torch.Generator().manual_seed(i)).int() for i in range(2))))
    half = lambda seed, *shape: torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16()  # noqa: E731
    rows = [place(half(i, 40, 128), half(100 + i, 40, 128)) for i in range(4)]
    weight, scale = (place(torch.rand(128), torch.rand(128) + 1) for _ in range(2))
    to, frm = place(ints(2, 3), ints(3, 2)), place(ints(0, 1), ints(1, -1))
    states, out = make_pool(torch, 90, 4, H, 128, 128), ints(2, 3).cuda()
    ws, big = g.new_workspace(0), torch.empty(g.gdn2_add_norm_bwd_workspace_bytes(40, 128), dtype=torch.uint8, device="cuda")

    def recurrent(a):
        p = states.clone()
        return lambda: (g.recurrent_fwd(*a["x"], p, a["slots"], out, a["cu"], index=a["index"], workspace=ws), p)

    def copies():
        p = states.clone()
        return lambda: (g.gdn2_state_copy(p, p, to, frm, workspace=ws), p)[1:]
    calls = [lambda: lambda: g.gated_norm_fwd(rows[0], rows[1], weight),
             lambda: lambda: g.gated_norm_bwd(rows[0], rows[1], weight, rows[2], workspace=big),
             lambda: lambda: g.add_norm_fwd(rows[0], rows[1], scale, weight),
             lambda: lambda: g.add_norm_bwd(rows[0], rows[1], scale, weight, rows[2], rows[3], workspace=big),
             lambda: lambda: g.tree_fwd(*args[12]["x"], states, args[12]["slots"], args[12]["cu"], args[12]["parents"], 8, workspace=ws),
             lambda: lambda: g.tree_fwd(*args[n]["x"], states, args[n]["slots"], args[n]["cu"], args[n]["parents"], 44, workspace=ws),
             lambda: recurrent(args[n]), copies]
    source, target = [ints(i).cuda() for i in range(2)], ints(2).cuda()
    flat = lambda r: [r] if torch.is_tensor(r) else list(r)  # noqa: E731
    for which, call in enumerate(calls):
        want = []
        for i in range(2):
            g.gdn2_state_copy(pool, pool, target, source[i], workspace=ws)
            torch.cuda.synchronize()
            want.append([a.clone() for a in flat(call()())])
            torch.cuda.synchronize()
        assert not all(torch.equal(a, b) for a, b in zip(*want))
        for turn in range(40):
            ready = call()                                         # what it copies it copies before
            g.gdn2_state_copy(pool, pool, target, source[turn % 2], workspace=ws)
            got = flat(ready())
            for a, b in zip(got, want[turn % 2]):
                if a.shape[0] in (12, n):                          # the second turn has one token fewer
                    a, b = a[:a.shape[0] - turn % 2], b[:b.shape[0] - turn % 2]
                assert torch.equal(a, b), (which, turn)
    assert g.gdn2_workspace_status(ws) == 0


def test_a_launch_that_fails_leaves_no_error_behind():
    """A launch on the legacy default stream is refused while a blocking stream is being captured.  The call says so, and
    the next call, of any kind, does not report it again."""
    torch, g = cuda_or_skip()
    from cuda.bindings import runtime as rt
    x, pool = tokens(torch, 70, 3, 2, 128, 128, "bf16"), make_pool(torch, 71, 3, 2, 128, 128)
    slots, other, cu, parents = (i32(torch, v) for v in ([0], [1], [0, 3], [-1, 0, 0]))
    o, gate, w = x[2].reshape(-1, 128), x[5].reshape(-1, 128), torch.ones(128, device="cuda")
    ws = g.new_workspace(g.gdn2_gated_norm_bwd_workspace_bytes(6, 128))
    out = [torch.empty_like(o) for _ in range(3)] + [torch.empty_like(w)]
    calls = [lambda: g.gdn2_tree_fwd(*x, pool, slots, cu, parents, x[2], 3, workspace=ws),
             lambda: g.gdn2_recurrent_fwd(*x, pool, slots, other, cu, None, x[2], workspace=ws),
             lambda: g.gdn2_state_copy(pool, pool, other, slots, workspace=ws),
             lambda: g.gdn2_gated_norm_fwd(o, gate, w, out[0]),
             lambda: g.gdn2_gated_norm_bwd(o, gate, w, gate, *out[1:], workspace=ws),
             lambda: g.gdn2_add_norm_fwd(o, gate, None, w, out[0], out[1])]
    torch.cuda.synchronize()
    assert torch.cuda.current_stream().cuda_stream == 0
    for call in calls:
        err, stream = rt.cudaStreamCreate()                       # a blocking one
        assert not err
        assert not rt.cudaStreamBeginCapture(stream, rt.cudaStreamCaptureMode.cudaStreamCaptureModeRelaxed)[0]
        try:
            with pytest.raises(g.GDN2Error):
                call()
        finally:
            rt.cudaStreamEndCapture(stream)                       # invalidated: an error, and no graph
            rt.cudaGetLastError()
            rt.cudaStreamDestroy(stream)
        g.gdn2_rms_norm(out[0], w)                                # a launcher that reports the last error it finds
        call()
    torch.cuda.synchronize()


def test_calls_of_every_kind_at_once():
    """Host threads with a stream each: trees on both kernels, runs, reorders, norms and the tensor-core prefill beside one
    another, all without a workspace of their own (the calls over slots share the device's status), give what each gives
    alone."""
    import threading
    torch, g = cuda_or_skip()
    H, n, B = 16, 44, 10
    rng = np.random.default_rng(1)
    x, few = tokens(torch, 100, n * B, H, 128, 128, "bf16"), tokens(torch, 101, 6 * B, H, 64, 128, "f32")
    pool, small = make_pool(torch, 102, 2 * B, H, 128, 128), make_pool(torch, 103, 2 * B, H, 64, 128)
    slots, other, cu = i32(torch, range(B)), i32(torch, range(B, 2 * B)), i32(torch, range(0, n * B + 1, n))
    cu6, par = i32(torch, range(0, 6 * B + 1, 6)), i32(torch, sum((random_tree(rng, n, 7) for _ in range(B)), []))
    par6 = i32(torch, sum((random_tree(rng, 6, 3) for _ in range(B)), []))
    perm, weight = rng.permutation(2 * B), torch.rand(128, device="cuda")
    to, frm = i32(torch, perm), i32(torch, np.roll(perm, 1))
    rows, dense = x[2].reshape(-1, 128), [a.view(B, n, H, 128) for a in x]

    def runs():
        p = pool.clone()
        return g.recurrent_fwd(*x, p, slots, other, cu), p

    def reorder():
        p = pool.clone()
        g.gdn2_state_copy(p, p, to, frm)
        return (p,)
    kinds = [lambda: (g.tree_fwd(*x, pool, slots, cu, par, n),), lambda: (g.tree_fwd(*few, small, slots, cu6, par6, 6),), runs, reorder,
             lambda: g.gated_norm_bwd(rows, x[5].reshape(-1, 128), weight, rows), lambda: g.chunk_fwd(*dense)]
    wants = [[a.clone() for a in kind()] for kind in kinds]
    torch.cuda.synchronize()
    g.gdn2_shared_status()
    wrong = []

    def work(kind, want):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(30):
                got = kind()
                stream.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want)):
                    wrong.append(kinds.index(kind))
    threads = [threading.Thread(target=work, args=pair) for pair in zip(kinds, wants)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong and g.gdn2_shared_status() == 0


def test_two_graphs_share_a_workspace():
    """The workspace of the calls over slots holds status words only: two captured graphs replayed at the same
    time on two streams do not disturb one another, and what either reports stays reported."""
    torch, g = cuda_or_skip()
    H, B = 2, 40
    ws, graphs, outs, wants = g.new_workspace(0), [], [], []
    torch.cuda.synchronize()
    for seed, last in ((60, B - 1), (61, 77)):           # the second one's last tree hangs on no slot
        x = tokens(torch, seed, 20 * B, H, 128, 128, "bf16")
        pool = make_pool(torch, seed, B, H, 128, 128)
        rng = np.random.default_rng(seed)
        par = sum((random_tree(rng, 20, 5) for _ in range(B)), [])
        slots = i32(torch, list(range(B - 1)) + [last])
        cu, parents = i32(torch, range(0, 20 * B + 1, 20)), i32(torch, par)
        o = torch.full_like(x[2], float("nan"))
        g.gdn2_tree_fwd(*x, pool, slots, cu, parents, o, 20)
        wants.append(o.clone())
        graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=s):
            g.gdn2_tree_fwd(*x, pool, slots, cu, parents, o, 20, workspace=ws)
        graphs.append((graph, s, x, pool, slots, cu, parents))
        outs.append(o)
    for _ in range(5):
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        for graph, s, *_ in graphs:
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], wants[0])
        assert torch.equal(outs[1].nan_to_num(7.0), wants[1].nan_to_num(7.0)) and torch.isnan(outs[1][-20:]).all()
        assert g.gdn2_workspace_status(ws, clear=True) == g.DEV_SLOT


def test_serving_round_together():
    """As a server uses them: fork a sequence, draft a tree for each continuation, read the tree out, norm and
    gate it, take the accepted paths into the cache, and move the survivors together; everything captured in
    one graph and replayed on new inputs, against the fp64 definitions."""
    torch, g = cuda_or_skip()
    H, K, V, n = 4, 128, 128, 12
    rng = np.random.default_rng(3)
    pool = make_pool(torch, 30, 8, H, K, V)
    x = tokens(torch, 31, 2 * n, H, K, V, "bf16")
    gate = torch.randn(2 * n, H, V, generator=torch.Generator().manual_seed(32)).bfloat16().cuda()
    weight = torch.ones(V, device="cuda")
    parents = i32(torch, random_tree(rng, n, 4) + random_tree(rng, n, 4))
    cu, slots = i32(torch, [0, n, 2 * n]), i32(torch, [6, 7])
    fork = i32(torch, [6, 7]), i32(torch, [2, 2])
    path_cu, path = i32(torch, [0, 2, 4]), i32(torch, [0, 0, n, n])
    pack = i32(torch, [0, 1, 6, 7]), i32(torch, [6, 7, -1, -1])
    o, y, ws = torch.empty_like(x[2]), torch.empty_like(x[2]), g.new_workspace(0)

    def round_():
        g.gdn2_state_copy(pool, pool, *fork, workspace=ws)
        g.gdn2_tree_fwd(*x, pool, slots, cu, parents, o, n, workspace=ws)
        g.gdn2_gated_norm_fwd(o, gate, weight, y)
        g.gdn2_recurrent_fwd(*x, pool, slots, slots, path_cu, path, None, workspace=ws)
        g.gdn2_state_copy(pool, pool, *pack, workspace=ws)

    keep = pool.clone()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        round_()
    for seed in (40, 41):
        pool.copy_(keep)
        for a, b in zip(x, tokens(torch, seed, 2 * n, H, K, V, "bf16")):
            a.copy_(b)
        par = random_tree(rng, n, 3), random_tree(rng, n, 6)
        parents.copy_(i32(torch, par[0] + par[1]))
        ends = [int(rng.integers(1, n)), int(rng.integers(1, n))]
        rows = [[max(0, p[e]), e] for p, e in zip(par, ends)]
        path.copy_(i32(torch, rows[0] + [n + r for r in rows[1]]))
        graph.replay()
        torch.cuda.synchronize()
        ref = f64(keep)
        ref[[6, 7]] = ref[2]
        xs = [f64(a) for a in x]
        ro = op.tree(*xs, ref, [6, 7], [0, n, 2 * n], par[0] + par[1])
        close(o, ro, "bf16")
        ry = op.gated_norm(f64(o), f64(gate), f64(weight))
        assert (np.abs(f64(y) - ry) <= (2.0 ** -8 + 2.0 ** -17) * np.abs(ry) + 1e-30).all()
        _, ref = op.recurrent(*xs, ref, [6, 7], [6, 7], [0, 2, 4], path.tolist())
        close(pool, op.state_copy(ref, ref, [0, 1, 6, 7], [6, 7, -1, -1]), "f32")
        assert g.gdn2_workspace_status(ws) == 0
