"""The gated linear recurrence (streams and packed rows), the group norm and the products in 8-bit integers on the GPU,
against float64 references with bounds derived from the arithmetic (tests/_gated_ref.py)."""
import numpy as np
import pytest
import torch

import selective_state_space_chunked_amd as ssm

from . import _gated_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
GATED_OUT = ("glam", "gr_bias", "gi_bias", "gh0", "h_last")   # float32 whatever the streams


def gen(seed):
    return np.random.default_rng(seed)


def dev(a, dtype="f32"):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DT[dtype]).to(DEV)


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


# ---------------------------------------------------------------------------
# gated recurrence over streams
# ---------------------------------------------------------------------------
def gated_inputs(B, D, L, dtype, r, state=True, bias=True, spread=1.0):
    t = {k: dev(spread * r.normal(size=(B, D, L)), dtype) for k in ("x", "r", "i")}
    t["lam"] = dev(np.log(np.expm1(-np.log(r.uniform(0.9, 0.999, D)))))
    t["r_bias"], t["i_bias"] = (dev(0.5 * r.normal(size=D)) if bias else None for _ in range(2))
    t["h0"] = dev(r.normal(size=(B, D))) if state else None
    gy = dev(r.normal(size=(B, D, L)), dtype)
    return t, gy, dev(r.normal(size=(B, D))) if state else None


def arrays(t):
    return [f64(t[k]) for k in ("x", "r", "i", "lam", "r_bias", "i_bias")]


def gated_check(t, gy, gl, dtype, power=8.0):
    f = ssm.gated_fwd(want_h_last=True, want_ckpt=True, power=power, **t)
    for k, (ref, err) in R.gated_fwd(*arrays(t), power, f64(t["h0"])).items():
        R.check(k, f[k], ref, err, "f32" if k in GATED_OUT else dtype)
    g = ssm.gated_bwd(gy=gy, gh_last=gl, ckpt=f["ckpt"], power=power, **t)
    assert set(g) == {"gx", "gr", "gi", "glam", "gr_bias", "gi_bias", "gh0"}
    for k, (ref, err) in R.gated_bwd(*arrays(t), power, f64(t["h0"]), f64(gy), f64(gl)).items():
        R.check(k, g[k], ref, err, "f32" if k in GATED_OUT else dtype)
    return f, g


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,D,L", [(1, 1, 1), (2, 3, 2), (3, 5, 7), (1, 17, 8), (2, 9, 9), (1, 4, 127), (2, 33, 128),
                                   (1, 3, 129), (2, 5, 512), (1, 6, 513), (3, 2, 1000), (1, 2, 2048), (2, 3, 2057),
                                   (1, 2, 8192), (1, 3, 9001), (1, 1, 20011)])
def test_gated(B, D, L, dtype):
    t, gy, gl = gated_inputs(B, D, L, dtype, gen(B + D + L), state=L % 2 == 1, bias=L % 3 != 0)
    gated_check(t, gy, gl, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,D,L", [(8, 2051, 299), (5, 900, 700), (3, 350, 2500), (3, 350, 130)])
def test_gated_many_rows(B, D, L, dtype):
    """Rows enough that 16, 64 and 256 lanes share one, over several tiles."""
    t, gy, gl = gated_inputs(B, D, L, dtype, gen(7))
    gated_check(t, gy, gl, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gated_views_and_outputs(dtype):
    """Streams that are slices and broadcasts, outputs in slices of wider buffers; what lies around them stays."""
    r = gen(3)
    B, D, L = 3, 5, 301
    t, gy, gl = gated_inputs(B, D, L, dtype, r)
    wide = {k: dev(r.normal(size=(B, D + 1, L + 9)), dtype) for k in ("x", "i", "gy")}
    t["x"], t["i"], gy = wide["x"][:, 1:, 3:3 + L], wide["i"][:, :D, 1:1 + L], wide["gy"][:, 1:, 8:8 + L]
    t["r"] = dev(r.normal(size=(B, 1, L)), dtype).expand(B, D, L)
    ref = R.gated_fwd(*arrays(t), 8.0, f64(t["h0"]))
    back = R.gated_bwd(*arrays(t), 8.0, f64(t["h0"]), f64(gy), f64(gl))
    bufs = {k: torch.full((D, B + 1, L + 7), 7.0, dtype=DT[dtype], device=DEV) for k in ("y", "gx", "gr", "gi")}
    outs = {k: b[:, :B, 2:2 + L].transpose(0, 1) for k, b in bufs.items()}   # channels outside the batch
    f = ssm.gated_fwd(want_ckpt=True, out={"y": outs["y"]}, **t)
    assert f["y"] is outs["y"]
    R.check("y", f["y"], *ref["y"], dtype)
    g = ssm.gated_bwd(gy=gy, gh_last=gl, ckpt=f["ckpt"], out={k: outs[k] for k in ("gx", "gr", "gi")}, **t)
    for k, v in back.items():
        R.check(k, g[k], *v, "f32" if k in GATED_OUT else dtype)
    for b in bufs.values():
        assert (b[:, B] == 7).all() and (b[:, :, :2] == 7).all() and (b[:, :, 2 + L:] == 7).all()


def test_gated_states_again_and_determinism():
    """Without the states the backward forms them again: the same bits.  Each wanted output alone: the same bits too."""
    t, gy, gl = gated_inputs(2, 33, 1300, "bf16", gen(4))
    f = ssm.gated_fwd(want_h_last=True, want_ckpt=True, **t)
    par = dict(gy=gy, gh_last=gl, **t)
    g, again = ssm.gated_bwd(ckpt=f["ckpt"], **par), ssm.gated_bwd(**par)
    for k in g:
        assert torch.equal(g[k], again[k]), k
        one = ssm.gated_bwd(ckpt=f["ckpt"], want=(k,), **par)
        assert list(one) == [k] and torch.equal(one[k], g[k]), k
    for k in ("y", "h_last", "ckpt"):
        one = ssm.gated_fwd(**t, want_y=k == "y", want_h_last=k == "h_last", want_ckpt=k == "ckpt")
        assert list(one) == [k] and torch.equal(one[k], f[k]), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gated_segments(dtype):
    """A stream in two calls, the state handed on: forward, and the gradients of the first with gh_last from the second."""
    t, gy, _ = gated_inputs(2, 7, 700, dtype, gen(5))
    whole = R.gated_bwd(*arrays(t), 8.0, f64(t["h0"]), f64(gy), None)
    y = R.gated_fwd(*arrays(t), 8.0, f64(t["h0"]))["y"]
    cut = 333
    part = [{**t, **{k: t[k][..., s] for k in ("x", "r", "i")}} for s in (slice(0, cut), slice(cut, None))]
    a = ssm.gated_fwd(want_h_last=True, want_ckpt=True, **part[0])
    part[1]["h0"] = a["h_last"]
    b = ssm.gated_fwd(want_ckpt=True, **part[1])
    R.check("y", torch.cat([a["y"], b["y"]], -1), y[0], 2 * y[1], dtype)
    gb = ssm.gated_bwd(gy=gy[..., cut:], ckpt=b["ckpt"], **part[1])
    ga = ssm.gated_bwd(gy=gy[..., :cut], gh_last=gb["gh0"], ckpt=a["ckpt"], **part[0])
    for k in ("gx", "gr", "gi"):
        R.check(k, torch.cat([ga[k], gb[k]], -1), whole[k][0], 2 * whole[k][1], dtype)
    for k in ("glam", "gr_bias", "gi_bias"):
        R.check(k, ga[k] + gb[k], whole[k][0], 2 * whole[k][1] + R.U * np.abs(f64(ga[k])), "f32")
    R.check("gh0", ga["gh0"], whole["gh0"][0], 2 * whole["gh0"][1], "f32")


def test_gated_gradient_by_differences():
    """Directional differences of the loss in float64, formed by the reference's forward alone."""
    r = gen(6)
    t, gy, gl = gated_inputs(2, 4, 150, "f32", r)
    g = ssm.gated_bwd(gy=gy, gh_last=gl, **t)
    names = {"gx": "x", "gr": "r", "gi": "i", "glam": "lam", "gr_bias": "r_bias", "gi_bias": "i_bias", "gh0": "h0"}
    base = {k: f64(v) for k, v in t.items()}

    def loss(v):
        f = R.gated_fwd(*(v[k] for k in ("x", "r", "i", "lam", "r_bias", "i_bias")), 8.0, v["h0"])
        return (f64(gy) * f["y"][0]).sum() + (f64(gl) * f["h_last"][0]).sum()

    for k, n in names.items():
        d = r.normal(size=base[n].shape)
        eps = 1e-5
        num = (loss({**base, n: base[n] + eps * d}) - loss({**base, n: base[n] - eps * d})) / (2 * eps)
        want = (f64(g[k]) * d).sum()
        # a central difference is off by about eps^2 times the third derivative, the gradient by fp32's errors
        assert abs(num - want) <= 1e-4 * np.linalg.norm(f64(g[k])) * np.linalg.norm(d), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gated_extremes(dtype):
    """Gates that are shut and wide open, slow and fast channels: finite, and the formula's values."""
    r = gen(8)
    B, D, L = 2, 6, 400
    t, gy, gl = gated_inputs(B, D, L, dtype, r, spread=4.0)
    t["r"][0, :, 50:60] = -80.0
    t["r"][1, :, 100:] = 30.0
    t["i"][0, :, 200:] = -60.0
    t["i"][1, :, :50] = 25.0
    t["lam"] = dev(np.array([-30.0, -12.0, -3.0, 0.0, 3.0, 25.0]))
    for power in (0.25, 8.0, 64.0):
        f, g = gated_check(t, gy, gl, dtype, power)
        assert all(torch.isfinite(v).all() for v in (*f.values(), *g.values()))
    # a gate below the exponential's range is shut: the state stays as it is, and nothing becomes NaN
    t["r"][:] = -200.0
    t["x"][:] = 1e30
    f = ssm.gated_fwd(want_h_last=True, want_ckpt=True, **t)
    assert torch.equal(f["h_last"], t["h0"])
    g = ssm.gated_bwd(gy=gy, gh_last=gl, ckpt=f["ckpt"], **t)
    for k in ("gx", "gr", "gi", "glam", "gr_bias", "gi_bias"):
        assert (g[k] == 0).all(), k


def test_gated_non_finite_values_stay_in_their_row():
    """A NaN or an infinity reaches the later steps of its row (and, backward, the earlier ones), no other row."""
    t, gy, gl = gated_inputs(2, 5, 300, "f32", gen(9))
    ref = ssm.gated_fwd(want_ckpt=True, **t)
    rg = ssm.gated_bwd(gy=gy, gh_last=gl, ckpt=ref["ckpt"], **t)
    for name, v in (("x", float("nan")), ("r", float("nan")), ("i", float("nan")), ("x", float("inf"))):
        u = {**t, name: t[name].clone()}
        u[name][1, 2, 297] = v
        f = ssm.gated_fwd(want_ckpt=True, want_h_last=True, **u)
        assert torch.equal(f["y"][1, 2, :297], ref["y"][1, 2, :297])
        assert not torch.isfinite(f["y"][1, 2, 297:]).any() and not torch.isfinite(f["h_last"][1, 2])
        g = ssm.gated_bwd(gy=gy, gh_last=gl, ckpt=f["ckpt"], **u)
        for k in ("gx", "gr", "gi"):
            keep = torch.ones(2, 5, dtype=torch.bool, device=DEV)
            keep[1, 2] = False
            assert torch.equal(g[k][keep], rg[k][keep]), (name, k)
            assert torch.isfinite(f["y"][keep]).all()
        if name != "r":   # the decay does not depend on x and i: mu is as it was
            assert torch.equal(g["gh0"], rg["gh0"])


@pytest.mark.parametrize("B,D,L", [(0, 3, 5), (2, 0, 5), (2, 3, 0)])
def test_gated_empty(B, D, L):
    t, gy, gl = gated_inputs(B, D, L, "bf16", gen(10))
    f = ssm.gated_fwd(want_h_last=True, want_ckpt=True, **t)
    assert f["y"].shape == (B, D, L) and torch.equal(f["h_last"], t["h0"])
    g = ssm.gated_bwd(gy=gy, gh_last=gl, **t)
    assert torch.equal(g["gh0"], gl)
    for k in ("glam", "gr_bias", "gi_bias"):
        assert g[k].shape == (D,) and (g[k] == 0).all()
    t["h0"] = None
    if L == 0:
        assert (ssm.gated_fwd(want_h_last=True, **t)["h_last"] == 0).all()


# ---------------------------------------------------------------------------
# gated recurrence over packed rows
# ---------------------------------------------------------------------------
def rows(T, D, dtype, r, view):
    """(T, D) values, as a slice of wider rows that do not start on a whole vector."""
    if not view:
        return dev(r.normal(size=(T, D)), dtype)
    return dev(r.normal(size=(T, D + 11)), dtype)[:, 3:3 + D]


def tok_inputs(T, D, dtype, r, view=False, bias=True):
    t = {k: rows(T, D, dtype, r, view) for k in ("x", "r", "i")}
    t["lam"] = dev(np.log(np.expm1(-np.log(r.uniform(0.9, 0.999, D)))))
    t["r_bias"], t["i_bias"] = (dev(0.5 * r.normal(size=D)) if bias else None for _ in range(2))
    return t


def tok_reference(t, start, slot, fresh, pool, y):
    """Sequence by sequence through the streams' reference: rows and slots, with bounds; what none owns stays."""
    x, r, i, lam, rb, ib = arrays(t)
    y, dy, pool, dpool = f64(y), np.zeros(y.shape), f64(pool), np.zeros(pool.shape)
    taken = set()
    for s in range(len(slot)):
        a, b = start[s], start[s + 1]
        if not 0 <= slot[s] < len(pool) or a >= b or slot[s] in taken:
            taken.add(slot[s])
            continue
        taken.add(slot[s])
        h0 = None if fresh is not None and fresh[s] else pool[slot[s]][None]
        f = R.gated_fwd(*(v[a:b].T[None] for v in (x, r, i)), lam, rb, ib, 8.0, h0)
        y[a:b], dy[a:b] = f["y"][0][0].T, f["y"][1][0].T
        pool[slot[s]], dpool[slot[s]] = f["h_last"][0][0], f["h_last"][1][0]
    return y, dy, pool, dpool


def tok_check(t, start, slot, fresh, slots, dtype, r, step=False):
    T, D = t["x"].shape
    whole = dev(r.normal(size=(slots + 2, D + 5)))
    pool = whole[1:-1, :D]
    wide = torch.full((T + 2, D + 9), 7.0, dtype=DT[dtype], device=DEV)
    y = wide[1:T + 1, 5:5 + D]
    ref = tok_reference(t, start, slot, fresh, pool, y)
    keep = whole.clone()
    at = dict(seq_start=None if step else torch.tensor(start, dtype=torch.int32, device=DEV),
              slot=torch.tensor(slot, dtype=torch.int32, device=DEV),
              fresh=None if fresh is None else torch.tensor(fresh, dtype=torch.bool, device=DEV))
    f = ssm.tokens_gated(pool=pool, out={"y": y}, **at, **t)
    assert f["y"] is y
    R.check("y", y, ref[0], ref[1], dtype)
    R.check("pool", pool, ref[2], ref[3], "f32")
    owned = ref[1].max(1) > 0
    assert (wide[0] == 7).all() and (wide[-1] == 7).all() and (wide[:, :5] == 7).all() and (wide[:, 5 + D:] == 7).all()
    assert (y[torch.from_numpy(~owned).to(DEV)] == 7).all()
    assert torch.equal(whole[0], keep[0]) and torch.equal(whole[-1], keep[-1]) and torch.equal(whole[:, D:], keep[:, D:])
    untouched = [k for k in range(slots) if not ref[3][k].any()]
    assert torch.equal(pool[untouched], keep[1:-1, :D][untouched])


LISTS = {
    "one": ([0, 100], [0], None, 1),
    "long": ([0, 1500], [1], [True], 3),
    "ragged": ([0, 1, 40, 40, 41, 300, 333], [3, 0, 5, 2, -1, 4], [True, False, True, False, False, True], 7),
    "gap behind": ([5, 90, 200], [1, 0], [False, True], 2),
    "same slot": ([0, 50, 100, 150], [1, 1, 0], [False, False, True], 2),
    "past the pool": ([0, 50, 100], [7, 1], None, 3),
}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,view", [(1, False), (3, True), (64, False), (258, True), (1028, False)])
@pytest.mark.parametrize("name", LISTS)
def test_tokens_gated(name, D, view, dtype):
    start, slot, fresh, slots = LISTS[name]
    r = gen(D + len(name))
    T = start[-1] + (13 if name == "gap behind" else 0)
    tok_check(tok_inputs(T, D, dtype, r, view, bias=D != 64), start, slot, fresh, slots, dtype, r)


def test_tokens_gated_many_ranges():
    """Ranges enough that a kernel of its own composes the states between them, in more than one turn of it."""
    r = gen(12)
    T, D = 9000, 40
    start = [0, 17, 4000, 4000, 8990, 9000]
    tok_check(tok_inputs(T, D, "f32", r), start, [2, 0, 4, 3, 1], [False, True, False, False, True], 5, "f32", r)


def test_tokens_gated_thousands_of_sequences():
    r = gen(13)
    n = r.integers(0, 5, 1500)
    start = [0, *np.cumsum(n)]
    slot = r.permutation(1600)[:1500]
    slot[r.integers(0, 1500, 60)] = -1
    tok_check(tok_inputs(int(start[-1]), 36, "bf16", r), [int(v) for v in start], [int(v) for v in slot],
              [bool(v) for v in r.random(1500) < 0.5], 1600, "bf16", r)


def test_tokens_gated_non_finite_values_stay_in_their_sequence():
    """A NaN or an infinity, in a row or in a state, reaches the later rows of its sequence and no other one, inside a
    tile of rows, across tiles and across rows that no sequence owns."""
    r = gen(15)
    T, D = 700, 70
    start, slot = [0, 5, 20, 310, 320, 600, 690], [0, 1, 2, -1, 3, 4]
    t = tok_inputs(T, D, "f32", r)
    at = dict(seq_start=torch.tensor(start, dtype=torch.int32, device=DEV),
              slot=torch.tensor(slot, dtype=torch.int32, device=DEV))
    first = dev(r.normal(size=(5, D)))
    pool = first.clone()
    ref = ssm.tokens_gated(pool=pool, out={"y": torch.zeros(T, D, device=DEV)}, **at, **t)["y"]
    for name, row, v in (("x", 25, float("inf")), ("r", 2, float("nan")), ("i", 300, float("nan")), ("r", 315, float("nan")),
                         ("x", 599, float("nan")), ("pool", 2, float("nan")), ("pool", 3, float("-inf")), ("r", 695, float("nan"))):
        u, p = dict(t), first.clone()
        if name == "pool":
            p[row] = v
            row, seq = start[row if row < 3 else 4], row if row < 3 else 4
        else:
            u[name] = t[name].clone()
            u[name][row] = v
            seq = max(k for k in range(6) if start[k] <= row)
        y = ssm.tokens_gated(pool=p, out={"y": torch.zeros(T, D, device=DEV)}, **at, **u)["y"]
        own = torch.zeros(T, dtype=torch.bool, device=DEV)
        if slot[seq] >= 0 and row < start[6]:
            own[row:start[seq + 1]] = True
            assert not torch.isfinite(y[own]).any() and not torch.isfinite(p[slot[seq]]).any(), (name, row)
            p[slot[seq]] = pool[slot[seq]]
        assert torch.equal(y[~own], ref[~own]) and torch.equal(p, pool), (name, row)


def test_tokens_gated_determinism():
    """Every call gives the same bits, whichever tiles of rows run at the same time, on an idle GPU and on a busy one."""
    r = gen(17)
    T, D = 8192, 600
    t = tok_inputs(T, D, "bf16", r)
    t["lam"] = dev(np.full(D, -9.0))
    at = dict(seq_start=torch.tensor([0, 300, T], dtype=torch.int32, device=DEV), slot=torch.tensor([1, 0], dtype=torch.int32, device=DEV))
    first = dev(r.normal(size=(2, D)))
    ref = None
    big = torch.randn(4096, 4096, device=DEV)
    for k in range(12):
        pool = first.clone()
        if k % 3 == 1:
            torch.cuda.synchronize()
        if k % 3 == 2:
            big @ big
        got = [ssm.tokens_gated(pool=pool, **at, **t)["y"], pool]
        ref = ref or got
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1]), k


def test_tokens_gated_slow_channels_over_many_tiles():
    """Channels that keep what they have, so that what a row brings is handed on from tile to tile to the last row, and
    many tiles of few channels, whose workgroups run at the same time."""
    r = gen(16)
    for T, D in ((20000, 3), (3000, 200)):
        t = tok_inputs(T, D, "f32", r)
        t["lam"] = dev(np.full(D, -14.0))
        tok_check(t, [0, T - 5, T], [1, 0], [False, True], 2, "f32", r)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S,D,view", [(1, 1, False), (3, 7, True), (64, 260, False), (130, 1030, True)])
def test_tokens_gated_step(S, D, view, dtype):
    r = gen(S + D)
    slot = [int(v) for v in r.permutation(S + 4)[:S]]
    if S > 2:
        slot[1], slot[2] = -1, S + 9
    if S > 60:
        slot[40] = slot[7]   # the later one is an empty place
    fresh = [bool(v) for v in r.random(S) < 0.3] if D != 7 else None
    tok_check(tok_inputs(S, D, dtype, r, view), list(range(S + 1)), slot, fresh, S + 4, dtype, r, step=True)


@pytest.mark.parametrize("many", [False, True])
def test_gated_lists_that_do_not_ascend_stay_inside_the_buffers(many):
    """seq_start, slot and fresh are not checked on the host: whatever they hold, nothing outside the rows of y and the
    slots of the pool is written (what the rows then hold is unspecified)."""
    r = gen(14)
    D, T, S = 40, 300, 90 if many else 6
    big = np.iinfo(np.int32)
    starts = [[250, 0, 10, 290, 20, 300, 0], [500, 600, -7, 40, big.max, big.min, 299], [big.max] * 7,
              [-3, 200, 100, 299, 298, 10, 1000], [300, 250, 200, 150, 100, 50, 0]]
    if many:
        starts = [r.integers(-50, 400, S + 1) for _ in range(4)] + [np.arange(S, -1, -1) * 4]
    wide = torch.full((T + 2, D + 9), 7.0, device=DEV)
    pool = torch.full((S + 2, D), 7.0, device=DEV)
    t = tok_inputs(T, D, "f32", r, view=True)
    for i, st in enumerate(starts):
        slot = r.integers(0, S, S)
        slot[i % S] = (big.max, big.min, S, -1)[i % 4]
        ssm.tokens_gated(pool=pool[1:-1], out={"y": wide[1:T + 1, 4:4 + D]},
                         seq_start=torch.tensor(np.asarray(st), dtype=torch.int32, device=DEV),
                         slot=torch.tensor(slot, dtype=torch.int32, device=DEV),
                         fresh=torch.tensor(r.integers(0, 256, S), dtype=torch.uint8, device=DEV), **t)
        torch.cuda.synchronize()
        assert (wide[0] == 7).all() and (wide[-1] == 7).all() and (wide[:, :4] == 7).all() and (wide[:, 4 + D:] == 7).all()
        assert (pool[0] == 7).all() and (pool[-1] == 7).all()


# ---------------------------------------------------------------------------
# group norm
# ---------------------------------------------------------------------------
def norm_inputs(T, C, dtype, r, view=False, gate=True, par=True):
    x = rows(T, C, dtype, r, view)
    x += dev(0.5 * r.normal(size=C), dtype)
    t = dict(x=x, z=rows(T, C, dtype, r, view) if gate else None)
    t["w"], t["bias"] = (dev(1 + 0.3 * r.normal(size=C)), dev(0.3 * r.normal(size=C))) if par else (None, None)
    return t, rows(T, C, dtype, r, view)


def norm_check(t, gy, groups, dtype, silu, eps=1e-5):
    f = ssm.group_norm_fwd(groups=groups, eps=eps, silu=silu, **t)
    g = ssm.group_norm_bwd(gy=gy, groups=groups, eps=eps, silu=silu, **t)
    ref = R.norm(f64(t["x"]), groups, f64(t["w"]), f64(t["bias"]), eps, silu, f64(t["z"]), f64(gy))
    assert {**f, **g}.keys() == ref.keys()
    for k, v in {**f, **g}.items():
        R.check(k, v, *ref[k], "f32" if k in ("gw", "gbias") else dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,G,per", [(1, 1, 1), (3, 5, 1), (7, 1, 3), (2, 3, 8), (9, 7, 16), (33, 64, 8), (5, 3, 65), (17, 2, 64),
                                     (4, 3, 130), (3, 1, 136), (11, 33, 40), (2, 2, 519), (3, 3, 520), (6, 1, 1024),
                                     (3, 2, 2056), (2, 1, 2501), (5, 1, 4096), (2, 2, 8192), (2, 1, 8191), (1500, 4, 24)])
@pytest.mark.parametrize("silu,gate", [(False, False), (True, False), (False, True), (True, True)])
def test_norm(T, G, per, silu, gate, dtype):
    t, gy = norm_inputs(T, G * per, dtype, gen(T + G + per), view=T % 2 == 1, gate=gate, par=G != 7)
    norm_check(t, gy, G, dtype, silu)


@pytest.mark.parametrize("T, G, per, dtype", [(2111, 31, 65, "f32"), (2111, 31, 65, "bf16"), (4099, 75, 14, "bf16"), (3001, 7, 27, "f32"),
                                              (16400, 3, 127, "f32"), (40001, 10, 11, "f32")])
def test_norm_many_rows_of_odd_groups(T, G, per, dtype):
    t, gy = norm_inputs(T, G * per, dtype, gen(T + G + per))
    norm_check(t, gy, G, dtype, True)


def test_norm_means_far_from_zero():
    """Groups whose mean is many times their spread: the statistics come from the differences to it."""
    r = gen(20)
    t, gy = norm_inputs(40, 256, "f32", r)
    t["x"] = t["x"] + 300.0
    norm_check(t, gy, 4, "f32", True)
    t["x"] = torch.full_like(t["x"], 3.0)     # no spread at all: y is the bias's
    y = ssm.group_norm_fwd(groups=4, w=t["w"], bias=t["bias"], x=t["x"])["y"]
    assert torch.equal(y, t["bias"].expand_as(y))


def test_norm_outputs_and_determinism():
    r = gen(21)
    T, C, G = 300, 96, 3
    t, gy = norm_inputs(T, C, "bf16", r)
    f = ssm.group_norm_fwd(groups=G, **t)["y"]
    g = ssm.group_norm_bwd(gy=gy, groups=G, **t)
    bufs = {k: torch.full((T + 2, C + 7), 7.0, dtype=torch.bfloat16, device=DEV) for k in ("y", "gx", "gz")}
    outs = {k: b[1:-1, 3:3 + C] for k, b in bufs.items()}
    assert torch.equal(ssm.group_norm_fwd(groups=G, out={"y": outs["y"]}, **t)["y"], f)
    h = ssm.group_norm_bwd(gy=gy, groups=G, out={k: outs[k] for k in ("gx", "gz")}, **t)
    for k in g:
        assert torch.equal(h[k], g[k]), k
        one = ssm.group_norm_bwd(gy=gy, groups=G, want=(k,), **t)
        assert list(one) == [k] and torch.equal(one[k], g[k]), k
    for b in bufs.values():
        assert (b[0] == 7).all() and (b[-1] == 7).all() and (b[:, :3] == 7).all() and (b[:, 3 + C:] == 7).all()
    bad = t["x"].clone()   # a NaN stays in its group
    bad[5, 40] = float("nan")
    y = ssm.group_norm_fwd(groups=G, **{**t, "x": bad})["y"]
    assert torch.isnan(y[5, 32:64]).all()
    y[5, 32:64] = f[5, 32:64]
    assert torch.equal(y, f)


def test_norm_gradient_by_differences():
    r = gen(22)
    t, gy = norm_inputs(6, 40, "f32", r)
    g = ssm.group_norm_bwd(gy=gy, groups=5, silu=True, **t)
    base = {k: f64(v) for k, v in t.items()}

    def loss(v):
        return (f64(gy) * R.norm(v["x"], 5, v["w"], v["bias"], 1e-5, True, v["z"])["y"][0]).sum()

    for k, n in {"gx": "x", "gz": "z", "gw": "w", "gbias": "bias"}.items():
        d = r.normal(size=base[n].shape)
        num = (loss({**base, n: base[n] + 1e-5 * d}) - loss({**base, n: base[n] - 1e-5 * d})) / 2e-5
        assert abs(num - (f64(g[k]) * d).sum()) <= 1e-4 * np.linalg.norm(f64(g[k])) * np.linalg.norm(d), k


@pytest.mark.parametrize("T,C", [(0, 12), (5, 0)])
def test_norm_empty(T, C):
    t, gy = norm_inputs(T, C, "bf16", gen(23))
    assert ssm.group_norm_fwd(groups=3, **t)["y"].shape == (T, C)
    g = ssm.group_norm_bwd(gy=gy, groups=3, **t)
    assert g["gx"].shape == (T, C) and (g["gw"] == 0).all() and (g["gbias"] == 0).all()


# ---------------------------------------------------------------------------
# products in 8-bit integers
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,K", [(1, 1), (3, 2), (5, 3), (2, 4), (7, 63), (9, 515), (4, 2048), (3, 2049), (5, 8193), (2, 20001),
                                 (600, 64)])
def test_pack8(T, K, dtype):
    r = gen(T + K)
    x = rows(T, K, dtype, r, K % 2 == 1)
    x *= dev(np.exp(3 * r.normal(size=(T, 1))), dtype)
    q, s = R.pack(f64(x))
    f = ssm.tokens_pack8(x)
    assert np.array_equal(f["x8"].cpu().numpy(), q) and np.array_equal(f["x8_scale"].cpu().numpy(), s)
    wide = torch.full((T + 2, K + 9), 7, dtype=torch.int8, device=DEV)
    ssm.tokens_pack8(x, out={"x8": wide[1:-1, 5:5 + K]})
    assert torch.equal(wide[1:-1, 5:5 + K], f["x8"])
    assert (wide[0] == 7).all() and (wide[-1] == 7).all() and (wide[:, :5] == 7).all() and (wide[:, 5 + K:] == 7).all()


def test_pack8_special_rows():
    x = torch.randn(8, 700, device=DEV)
    x[0] = 0
    x[1] = 2.0 ** -101
    x[2, 5] = float("inf")
    x[3, 6] = float("nan")
    x[4, 9] = torch.finfo(torch.float32).max
    x[5, 699] = -1e30
    q, s = R.pack(f64(x))
    f = ssm.tokens_pack8(x)
    assert np.array_equal(f["x8"].cpu().numpy(), q) and np.array_equal(f["x8_scale"].cpu().numpy(), s, equal_nan=True)
    w = torch.ones(3, 700, dtype=torch.int8, device=DEV)
    # (in float32: the largest float is past bfloat16's)
    y = ssm.tokens_mm8(x8=f["x8"], x8_scale=f["x8_scale"], w8=w, w8_scale=torch.ones(3, device=DEV), dtype=torch.float32)["y"]
    assert torch.isnan(y[2:4]).all() and torch.isfinite(y[[0, 1, 4, 5, 6, 7]]).all() and (y[:2] == 0).all()


def mm8_inputs(T, K, N, r, view=False, bias=True):
    def bytes_(n):
        b = torch.from_numpy(r.integers(-128, 128, (n, K + 13)).astype(np.int8)).to(DEV)
        return b[:, 5:5 + K] if view else b[:, :K].contiguous()

    return dict(x8=bytes_(T), x8_scale=dev(r.uniform(0.01, 1, T)), w8=bytes_(N), w8_scale=dev(r.uniform(0.01, 1, N)),
                bias=dev(r.normal(size=N)) if bias else None)


def mm8_check(t, dtype, **kw):
    got = ssm.tokens_mm8(dtype=DT[dtype], **t, **kw)["y"]
    v = {k: None if a is None else a.cpu().numpy() for k, a in t.items()}
    ref, err = R.mm8(v["x8"], v["x8_scale"], v["w8"], v["w8_scale"], None if v["bias"] is None else v["bias"].astype(np.float64))
    R.check("y", got, ref, err, dtype)
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [1, 3, 15, 16, 17, 64, 100, 127, 128, 129, 144, 240, 400, 515, 1024, 1100, 1152, 2032])
@pytest.mark.parametrize("T,N", [(1, 1), (2, 17), (16, 16), (17, 33), (40, 30), (64, 250), (65, 63), (130, 129), (300, 5)])
def test_mm8(T, N, K, dtype):
    r = gen(T + N + K)
    mm8_check(mm8_inputs(T, K, N, r, view=(T + K) % 2 == 1, bias=N % 2 == 1), dtype)


@pytest.mark.parametrize("T,K,N", [(2100, 640, 2000), (2049, 384, 4100), (1000, 200, 8200), (512, 4096, 512), (4096, 256, 264),
                                   (70, 8192, 500), (200, 131071, 40), (4000, 192, 3900), (3800, 64, 3700), (4096, 128, 4352), (4100, 384, 4300), (70000, 256, 128),
                                   (65664, 128, 64), (65664, 384, 61), (1030, 256, 1000), (1030, 208, 1000),
                                   (4096, 16, 4352), (4096, 336, 4352), (70000, 80, 128), (65664, 176, 64)])
def test_mm8_large(T, K, N):
    mm8_check(mm8_inputs(T, K, N, gen(31)), "bf16")
    mm8_check(mm8_inputs(T, K, N, gen(32), view=True), "f32")


def test_mm8_largest_sums():
    """The largest sum there is, 131071 products of (-128)^2, and its opposite."""
    K = 131071
    x = torch.full((70, K), -128, dtype=torch.int8, device=DEV)
    w = torch.full((3, K), -128, dtype=torch.int8, device=DEV)
    w[1] = 127
    one = torch.ones(70, device=DEV)
    for T in (1, 70):
        y = ssm.tokens_mm8(x8=x[:T], x8_scale=one[:T], w8=w, w8_scale=one[:3], dtype=torch.float32)["y"]
        assert torch.equal(y[:, 0], torch.full((T,), float(np.float32(K * 16384)), device=DEV))
        assert torch.equal(y[:, 1], torch.full((T,), float(np.float32(-K * 16256)), device=DEV))


def test_mm8_outputs_and_empty():
    r = gen(33)
    t = mm8_inputs(90, 200, 77, r)
    ref = mm8_check(t, "bf16")
    wide = torch.full((92, 90), 7.0, dtype=torch.bfloat16, device=DEV)
    y = ssm.tokens_mm8(out={"y": wide[1:-1, 3:80]}, **t)["y"]
    assert torch.equal(y, ref)
    assert (wide[0] == 7).all() and (wide[-1] == 7).all() and (wide[:, :3] == 7).all() and (wide[:, 80:] == 7).all()
    none = {**t, "x8": t["x8"][:, :0].contiguous(), "w8": t["w8"][:, :0].contiguous()}
    y = ssm.tokens_mm8(dtype=torch.float32, **none)["y"]   # no inputs: the bias
    assert torch.equal(y, t["bias"].expand_as(y))
    assert ssm.tokens_mm8(**{**t, "x8": t["x8"][:0], "x8_scale": t["x8_scale"][:0]})["y"].shape == (0, 77)
    f = ssm.tokens_pack8(torch.zeros(4, 0, device=DEV))
    assert f["x8"].shape == (4, 0) and (f["x8_scale"] == 0).all()
    assert ssm.tokens_pack8(torch.zeros(0, 9, device=DEV))["x8"].shape == (0, 9)


# ---------------------------------------------------------------------------
# together, on streams, in graphs, through both ways of the binding
# ---------------------------------------------------------------------------
def quantised(w):
    q, s = R.pack(w)
    return torch.from_numpy(q).to(DEV), dev(s)


def serving_weights(E, D, r):
    """A layer's projections in 8 bits (input and the two gates; output), its convolution, recurrence and norm."""
    p = {k: quantised(r.normal(size=(D, E)) / np.sqrt(E)) for k in ("x", "r", "i", "z")}
    p["o"] = quantised(r.normal(size=(E, D)) / np.sqrt(D))
    p["conv"], p["cbias"] = dev(r.normal(size=(D, 4)) / 2), dev(0.1 * r.normal(size=D))
    p["lam"] = dev(np.log(np.expm1(-np.log(r.uniform(0.9, 0.999, D)))))
    p["w"], p["b"] = dev(1 + 0.1 * r.normal(size=D)), dev(0.1 * r.normal(size=D))
    return p


def serve(p, rows, cpool, pool, where, dtype, groups):
    """rows -> 8 bits -> projections -> convolution -> gated recurrence -> gated norm -> 8 bits -> output projection."""
    q = ssm.tokens_pack8(rows)
    at = dict(x8=q["x8"], x8_scale=q["x8_scale"], dtype=dtype)
    x, r, i, z = (ssm.tokens_mm8(w8=p[k][0], w8_scale=p[k][1], **at)["y"] for k in ("x", "r", "i", "z"))
    u = ssm.tokens_conv(x=x, w=p["conv"], bias=p["cbias"], silu=True, pool=cpool, **where)["y"]
    h = ssm.tokens_gated(x=u, r=r, i=i, lam=p["lam"], pool=pool, **where)["y"]
    y = ssm.group_norm_fwd(x=h, groups=groups, w=p["w"], bias=p["b"], z=z)["y"]
    q = ssm.tokens_pack8(y)
    return ssm.tokens_mm8(x8=q["x8"], x8_scale=q["x8_scale"], w8=p["o"][0], w8_scale=p["o"][1], dtype=dtype)["y"]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompts_then_tokens_of_a_gated_layer(dtype):
    """A whole serving layer over prompts and then token by token against the same layer in float64, every stage taking
    the stage before as the GPU rounded it; and each token alone gives what the token inside a prompt gives."""
    r = gen(40)
    E, D, G, lens = 96, 160, 5, [70, 1, 133]
    p = serving_weights(E, D, r)
    S, start = len(lens), [0, *np.cumsum(lens)]
    T = int(start[-1])
    rows = dev(r.normal(size=(T, E)), dtype)
    slot = torch.tensor([2, 0, 3], dtype=torch.int32, device=DEV)
    pools = [torch.zeros(5, D, 3, dtype=DT[dtype], device=DEV), torch.zeros(5, D, device=DEV)]
    where = dict(seq_start=torch.tensor(start, dtype=torch.int32, device=DEV), slot=slot,
                 fresh=torch.ones(S, dtype=torch.bool, device=DEV))
    whole = serve(p, rows, *pools, where, DT[dtype], G)
    ends = [v.clone() for v in pools]
    # the prompts but for their last five tokens, then those one by one
    cut = [max(n - 5, 0) for n in lens]
    take = torch.cat([torch.arange(start[s], start[s] + cut[s]) for s in range(S)]).to(DEV)
    pools = [torch.zeros_like(v) for v in pools]
    where["seq_start"] = torch.tensor([0, *np.cumsum(cut)], dtype=torch.int32, device=DEV)
    first = serve(p, rows[take].contiguous(), *pools, where, DT[dtype], G)
    same = [(first, whole[take])]
    for k in range(5):
        live = [s for s in range(S) if k >= 5 - min(lens[s], 5)]
        one = dict(slot=torch.tensor([int(slot[s]) if s in live else -1 for s in range(S)], dtype=torch.int32, device=DEV),
                   fresh=torch.tensor([lens[s] <= 5 and k == 5 - lens[s] for s in range(S)], device=DEV))
        at = torch.tensor([start[s + 1] - 5 + k if s in live else 0 for s in range(S)], device=DEV)
        # (places that are empty keep what the tensors they come in hold: those are given)
        x8 = ssm.tokens_pack8(rows[at].contiguous())
        g = {n: ssm.tokens_mm8(x8=x8["x8"], x8_scale=x8["x8_scale"], w8=p[n][0], w8_scale=p[n][1], dtype=DT[dtype])["y"]
             for n in ("x", "r", "i", "z")}
        zero = {"y": torch.zeros(S, D, dtype=DT[dtype], device=DEV)}
        u = ssm.tokens_conv(x=g["x"], w=p["conv"], bias=p["cbias"], silu=True, pool=pools[0], out=zero, **one)["y"]
        h = ssm.tokens_gated(x=u, r=g["r"], i=g["i"], lam=p["lam"], pool=pools[1], out={"y": torch.zeros_like(u)}, **one)["y"]
        y = ssm.group_norm_fwd(x=h, groups=G, w=p["w"], bias=p["b"], z=g["z"])["y"]
        q = ssm.tokens_pack8(y)
        o = ssm.tokens_mm8(x8=q["x8"], x8_scale=q["x8_scale"], w8=p["o"][0], w8_scale=p["o"][1], dtype=DT[dtype])["y"]
        same.append((o[live], whole[at[live]]))
    # The two ways differ by what fp32 rounds along a scan (or the next value of bf16), and so by a step of 8 bits here and
    # there: of at most 1/127 of a row's largest magnitude in each of D terms, added with random signs.
    for a, b in same:
        a, b = a.double(), b.double()
        assert float((a - b).norm() / b.norm()) < (2e-3 if dtype == "f32" else 2e-2)
    for a, b in zip(pools, ends):
        assert float((a.double() - b.double()).norm() / b.double().norm()) < (1e-5 if dtype == "f32" else 2e-2)
    # stage by stage against the references
    q = ssm.tokens_pack8(rows)
    v = {k: ssm.tokens_mm8(x8=q["x8"], x8_scale=q["x8_scale"], w8=p[k][0], w8_scale=p[k][1], dtype=DT[dtype])["y"] for k in "xriz"}
    x8, xs = q["x8"].cpu().numpy(), q["x8_scale"].cpu().numpy()
    for k in "xriz":
        R.check(k, v[k], *R.mm8(x8, xs, p[k][0].cpu().numpy(), p[k][1].cpu().numpy(), None), dtype)
    t = dict(x=v["x"], r=v["r"], i=v["i"], lam=p["lam"], r_bias=None, i_bias=None)
    tok_check(t, [int(s) for s in start], [2, 0, 3], [True] * 3, 5, dtype, r)
    h = ssm.gated_fwd(**{k: a.T.contiguous()[None] if k in "xri" else a for k, a in t.items()})["y"][0].T.contiguous()
    n = dict(x=h, z=v["z"], w=p["w"], bias=p["b"])
    norm_check(n, dev(r.normal(size=(T, D)), dtype), G, dtype, False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_training_step_of_a_gated_layer(dtype):
    """Convolution, gated recurrence and norm forward and back: the gradients that arrive at the input and at every
    parameter, against differences of the layer's loss in float64 and, stage by stage, against the references."""
    from . import _layer_ref as C
    r = gen(41)
    B, D, L, G, W = 2, 24, 200, 3, 4
    x = dev(r.normal(size=(B, D, L)), dtype)
    gates = {k: dev(r.normal(size=(B, D, L)), dtype) for k in "ri"}
    z, gy = dev(r.normal(size=(B * L, D)), dtype), dev(r.normal(size=(B * L, D)), dtype)
    w, cb = dev(r.normal(size=(D, W)) / 2), dev(0.1 * r.normal(size=D))
    lam = dev(np.log(np.expm1(-np.log(r.uniform(0.9, 0.999, D)))))
    nw, nb = dev(1 + 0.1 * r.normal(size=D)), dev(0.1 * r.normal(size=D))
    rows = lambda t: t.transpose(1, 2).reshape(B * L, D).contiguous()                      # noqa: E731
    streams = lambda t: t.reshape(B, L, D).transpose(1, 2).contiguous()                    # noqa: E731
    f = ssm.conv_fwd(x=x, w=w, bias=cb, silu=True, want_ckpt8=True)
    rec = dict(x=f["y"], lam=lam, **gates)
    h = ssm.gated_fwd(want_ckpt=True, **rec)
    n = dict(x=rows(h["y"]), groups=G, w=nw, bias=nb, z=z)
    y = ssm.group_norm_fwd(**n)["y"]
    gn = ssm.group_norm_bwd(gy=gy, **n)
    gr = ssm.gated_bwd(gy=streams(gn["gx"]), ckpt=h["ckpt"], **rec)
    gc = ssm.conv_bwd(gy=gr["gx"], x=x, w=w, bias=cb, silu=True)
    v, err, _ = C.conv_fwd(f64(x), f64(w), f64(cb), None, True)
    R.check("u", f["y"], v, err, dtype)
    a = [f64(f["y"]), f64(gates["r"]), f64(gates["i"]), f64(lam), None, None]
    R.check("h", h["y"], *R.gated_fwd(*a, 8.0, None)["y"], dtype)
    ref = R.norm(f64(n["x"]), G, f64(nw), f64(nb), 1e-5, False, f64(z), f64(gy))
    for k, g in {"y": y, **gn}.items():
        R.check(k, g, *ref[k], "f32" if k in ("gw", "gbias") else dtype)
    for k, v in R.gated_bwd(*a, 8.0, None, f64(streams(gn["gx"])), None).items():
        R.check(k, gr[k], *v, "f32" if k in GATED_OUT else dtype)

    def loss(x, w, cb, r_, i_, lam, nw, nb, z):
        u, _, _ = C.conv_fwd(x, w, cb, None, True)
        h = R.gated_fwd(u, r_, i_, lam, None, None, 8.0, None)["y"][0]
        return (f64(gy) * R.norm(h.transpose(0, 2, 1).reshape(B * L, D), G, nw, nb, 1e-5, False, z)["y"][0]).sum()

    base = [f64(v) for v in (x, w, cb, gates["r"], gates["i"], lam, nw, nb, z)]
    got = [gc["gx"], gc["gw"], gc["gbias"], gr["gr"], gr["gi"], gr["glam"], gn["gw"], gn["gbias"], gn["gz"]]
    for k, g in enumerate(got):
        d = r.normal(size=base[k].shape)
        far = [[v + s * 1e-5 * d if j == k else v for j, v in enumerate(base)] for s in (1, -1)]
        num = (loss(*far[0]) - loss(*far[1])) / 2e-5
        # streams between the stages are rounded to their type: relative to the gradient's size that many half steps, and
        # the chain is three stages long, forward and back
        assert abs(num - (f64(g) * d).sum()) <= 12 * R.HALF[dtype] * np.linalg.norm(f64(g)) * np.linalg.norm(d) + \
            1e-4 * np.linalg.norm(f64(g)) * np.linalg.norm(d), k


def every_call(seed):
    """Every function of this file once, with plain tensors: a function that runs them on the same buffers again, and the
    buffers that other inputs may be copied to."""
    r = gen(seed)
    D, T, S = 72, 300, 5
    t, gy, gl = gated_inputs(2, 9, 1100, "bf16", r)
    tok = tok_inputs(T, D, "bf16", r)
    start = torch.tensor([0, 3, 3, 140, 290, 300], dtype=torch.int32, device=DEV)
    slot = torch.tensor([4, 1, -1, 0, 6], dtype=torch.int32, device=DEV)
    fresh = torch.tensor([0, 1, 0, 1, 0], dtype=torch.bool, device=DEV)
    keep, pool = dev(r.normal(size=(7, D))), torch.empty(7, D, device=DEV)
    n, ngy = norm_inputs(333, 64, "bf16", r)
    m = mm8_inputs(70, 256, 96, r)
    xr = dev(r.normal(size=(70, 256)), "bf16")

    def run():
        o = {}

        def put(name, d):
            o.update({f"{name} {k}": v for k, v in d.items()})
            return d

        f = put("gated", ssm.gated_fwd(want_h_last=True, want_ckpt=True, **t))
        put("gated bwd", ssm.gated_bwd(gy=gy, gh_last=gl, ckpt=f["ckpt"], **t))
        put("gated some", ssm.gated_bwd(gy=gy, want=("gi", "glam"), **t))
        pool.copy_(keep)
        put("tokens", ssm.tokens_gated(pool=pool, seq_start=start, slot=slot, fresh=fresh,
                                       out={"y": torch.zeros(T, D, dtype=torch.bfloat16, device=DEV)}, **tok))
        put("step", ssm.tokens_gated(pool=pool, slot=slot, **{k: v[:S] if k in "xri" else v for k, v in tok.items()},
                                     out={"y": torch.zeros(S, D, dtype=torch.bfloat16, device=DEV)}))
        o["pool"] = pool.clone()
        put("norm", ssm.group_norm_fwd(groups=4, silu=True, **n))
        put("norm bwd", ssm.group_norm_bwd(gy=ngy, groups=4, silu=True, **n))
        put("norm some", ssm.group_norm_bwd(gy=ngy, groups=2, want=("gx",), x=n["x"]))
        q = put("pack", ssm.tokens_pack8(xr))
        put("mm8", ssm.tokens_mm8(**m))
        put("mm8 f32", ssm.tokens_mm8(**{**m, **q}, dtype=torch.float32))
        put("mm8 few", ssm.tokens_mm8(**{**m, "x8": m["x8"][:3], "x8_scale": m["x8_scale"][:3]}))
        return o

    return run, [t["x"], t["r"], gy, tok["x"], tok["i"], keep, n["x"], n["z"], ngy, xr]


def test_gated_streams_and_graphs():
    """Calls on a stream of their own, and captured calls replayed with other inputs, eager work and waits between them:
    every replay equals the eager call bit for bit."""
    run, buffers = every_call(50)
    ref = run()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        own = run()
    torch.cuda.synchronize()
    for k in ref:
        assert torch.equal(ref[k], own[k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = run()
    r = gen(51)
    for i in range(4):
        for b in buffers:
            b.copy_(torch.from_numpy(r.normal(size=tuple(b.shape))))
        graph.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in cap.items()}
        eager = run()
        torch.cuda.synchronize()
        for k in eager:
            assert torch.equal(eager[k], got[k]), (i, k)


def test_gated_native_calls_are_the_bindings():
    """Without an installed allocator plain calls go through the native module: the same keys and the same bits."""
    a = every_call(52)[0]()
    ssm.set_allocator(None)
    from selective_state_space_chunked_amd import binding
    made = []
    orig = binding._done

    def count(r):
        made.append(r is not NotImplemented)
        return orig(r)

    binding._done = count
    try:
        b = every_call(52)[0]()
    finally:
        binding._done = orig
    assert made and all(made)
    assert a.keys() == b.keys()
    for k in a:
        assert a[k].dtype == b[k].dtype and a[k].shape == b[k].shape and torch.equal(a[k], b[k]), k


def test_gated_native_calls_refuse_as_the_binding():
    """Arguments the native module leaves alone raise the binding's errors; those the library refuses, the library's."""
    ssm.set_allocator(None)
    x, lam = torch.zeros(2, 3, 10, device=DEV), torch.zeros(3, device=DEV)
    rows, i8 = torch.zeros(6, 3, device=DEV), dict(dtype=torch.int8, device=DEV)
    g, k = dict(x=x, r=x, i=x, lam=lam), dict(x=rows, r=rows, i=rows, lam=lam)
    m = dict(x8=torch.zeros(4, 6, **i8), x8_scale=torch.zeros(4, device=DEV), w8=torch.zeros(3, 6, **i8),
             w8_scale=torch.zeros(3, device=DEV))
    err = ssm.binding.SSMError
    for f, kw, exc in ((ssm.gated_fwd, dict(g, power=-1.0), err), (ssm.gated_fwd, dict(g, power=-1), err),
                       (ssm.gated_fwd, dict(g, power=1e60), err), (ssm.gated_fwd, dict(g, lam=torch.zeros(2, device=DEV)), ValueError),
                       (ssm.gated_fwd, dict(g, r=x.double()), TypeError), (ssm.gated_fwd, dict(g, lam=lam.cpu()), ValueError),
                       (ssm.gated_bwd, dict(g, gy=x[..., :9]), ValueError), (ssm.gated_bwd, dict(g, gy=x, want=("gz",)), ValueError),
                       (ssm.gated_bwd, dict(g, gy=x, ckpt=torch.zeros(2, 3, 2, device=DEV)), ValueError),
                       (ssm.tokens_gated, dict(k, pool=torch.zeros(4, 3, device=DEV)), err),           # 6 rows, 4 slots
                       (ssm.tokens_gated, dict(k, pool=torch.zeros(6, 3, 1, device=DEV)), ValueError),
                       (ssm.tokens_gated, dict(k, pool=torch.zeros(6, 3, device=DEV), out={"y": rows}), err),   # y over x
                       (ssm.group_norm_fwd, dict(x=rows, groups=2), err), (ssm.group_norm_fwd, dict(x=rows, groups=3, eps=-1.0), err),
                       (ssm.group_norm_fwd, dict(x=rows, groups="3"), TypeError),
                       (ssm.group_norm_bwd, dict(gy=rows, x=rows, groups=3, want=("gz",)), err),       # no z
                       (ssm.group_norm_bwd, dict(gy=rows[:5], x=rows, groups=3), ValueError),
                       (ssm.tokens_pack8, dict(x=rows.half()), TypeError),
                       (ssm.tokens_mm8, dict(m, w8=torch.zeros(3, 5, **i8)), ValueError),
                       (ssm.tokens_mm8, dict(m, x8_scale=None), ValueError),
                       (ssm.tokens_mm8, dict(m, dtype=torch.float64), TypeError)):
        with pytest.raises(exc):
            f(**kw)


def test_gated_offsets_past_32_bits():
    """Rows, streams and slots of wide strides, so that they lie past 2^32 bytes: as the same tensors laid out densely."""
    r = gen(60)
    T, D, S = 70, 24, 3
    wide, wide_out = (torch.empty(T * 2**26, dtype=torch.bfloat16, device=DEV) for _ in range(2))

    def spread(v, at):
        o = wide.as_strided(v.shape, (2**26 - 1, 1), at)
        o.copy_(v)
        return o

    t = tok_inputs(T, D, "bf16", r)
    far = {k: spread(t[k], 100 * n) for n, k in enumerate("xri")}
    out = wide_out.as_strided((T, D), (2**26 - 1, 1), 900)
    at = dict(seq_start=torch.tensor([0, 33, 34, T], dtype=torch.int32, device=DEV),
              slot=torch.tensor([2, 0, 1], dtype=torch.int32, device=DEV))
    first = torch.randn(S, D, device=DEV)
    base = torch.empty(2 * (2**30 + 4) + D, device=DEV)
    res = []
    for f in (False, True):
        for step in (False, True):
            pool = base.as_strided(first.shape, (2**30 + 4, 1)) if f else torch.empty_like(first)
            pool.copy_(first)
            a = {k: v[:S] if step and k in far else v for k, v in ({**t, **far} if f else t).items()}
            y = ssm.tokens_gated(pool=pool, out={"y": out[:len(a["x"])]} if f else {}, **a,
                                 **(dict(slot=at["slot"]) if step else at))["y"]
            res += [y.clone(), pool.clone()]
    for p, q in zip(res[:4], res[4:]):
        assert torch.equal(p, q)
    del base, pool
    n = dict(groups=3, w=dev(r.normal(size=D)), silu=True)
    dense, wide_ = dict(x=t["x"], z=t["r"], **n), dict(x=far["x"], z=far["r"], **n)
    assert torch.equal(ssm.group_norm_fwd(out={"y": out}, **wide_)["y"], ssm.group_norm_fwd(**dense)["y"])
    p, q = ssm.group_norm_bwd(gy=t["i"], **dense), ssm.group_norm_bwd(gy=far["i"], out={"gx": out}, **wide_)
    assert all(torch.equal(p[k], q[k]) for k in p)
    b8, out8 = wide.view(torch.int8), wide_out.view(torch.int8).as_strided((T, D), (2**26 + 3, 1), 900)
    p, q = ssm.tokens_pack8(t["x"]), ssm.tokens_pack8(far["x"], out={"x8": out8})
    assert all(torch.equal(p[k], q[k]) for k in p)
    for rows_, K in ((T, 40), (20, 128), (T, 128)):
        m = mm8_inputs(rows_, K, 50, r)
        w8 = b8.as_strided((50, K), (2**27, 1), 2**26)
        x8 = out8.as_strided((rows_, K), (2**26, 1), 16)
        w8.copy_(m["w8"])
        x8.copy_(m["x8"])
        ref = ssm.tokens_mm8(**m)["y"]
        assert torch.equal(ssm.tokens_mm8(**{**m, "w8": w8, "x8": x8})["y"], ref)
    x = {k: dev(r.normal(size=(2, 3, 700)), "bf16") for k in ("x", "r", "i", "gy")}
    g = {k: wide.as_strided((2, 3, 700), (2**32, 2**20, 1), 5000 * n) for n, k in enumerate(x)}
    for k in g:
        g[k].copy_(x[k])
    fo = wide_out.as_strided((2, 3, 700), (2**32, 2**20, 1), 3)
    lam = t["lam"][:3].contiguous()
    a = ssm.gated_bwd(lam=lam, **x)
    b = ssm.gated_bwd(lam=lam, out={"gr": fo}, **g)
    assert all(torch.equal(a[k], b[k]) for k in a)
    assert torch.equal(ssm.gated_fwd(lam=lam, **{k: v for k, v in g.items() if k != "gy"}, out={"y": fo})["y"],
                       ssm.gated_fwd(lam=lam, **{k: v for k, v in x.items() if k != "gy"})["y"])
