"""The AdamW step and the gradient clipping over a list of tensors, against the
fp64 oracle (oracle/adamw_oracle.py).

Bounds.  u = 2^-24 is the largest relative error of one rounding to float32, h = 2^-8 of one to
bfloat16.  All tests compare elementwise with a count of roundings:
  norm    sixteen squares are added in 32 bits: each square is rounded with the addition (fma), so the
          sum of a group is off by at most 16 u, and the norm by 8 u, and 1 u for its own rounding: 10 u
  factor  norm's 8 u and its rounding: 9 u; times g: 10 u for the clipped gradient (0 without clipping)
  m       b1 and 1 - b1 rounded (u each), the products (u each), their sum (u):
          u (2 |b1 m| + (2 + 10) |(1 - b1) g| + |m'|), without clipping 2 in place of 2 + 10
  v       1 - b2 or b2 (1), two products or one (2), with 8 bits the square v starts from (1), the sum (1),
          g twice (20): all terms positive, 6 u v' and 20 u with clipping
  r       half of v's and the root's own: 4 u, and 10 u with clipping
  step    lr/(1-b1^t) (1), 1/sqrt(1-b2^t) (1), eps (1), the fma (1), the fast division (2 units in the last
          place: 4), the product (1): 9 u of it, r's part, and m's error times its factor
  w       shrink (1) and the last fma (1): u (|w| + |w'|) on top
Second-order terms are covered by a last factor of 1.01.
"""
import ctypes as C
import math
import os

import numpy as np
import pytest

from oracle import adamw_oracle as O
from shampoo_second_order_b200 import _lib as L

U = 2.0 ** -24
FLT_MAX = float(np.finfo(np.float32).max)
B1, B2, EPS = 0.9, 0.999, 1e-8

torch = pytest.importorskip("torch")


# --------------------------------------------------------------------------
# CPU: the oracle's own pins
# --------------------------------------------------------------------------
def test_oracle_adamw_matches_torch_in_64_bits():
    rng = np.random.default_rng(1)
    w = rng.standard_normal(50)
    p = torch.nn.Parameter(torch.from_numpy(w.copy()))
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(B1, B2), eps=EPS, weight_decay=0.03)
    m, v = np.zeros(50), np.zeros(50)
    for t in range(1, 6):
        g = rng.standard_normal(50)
        p.grad = torch.from_numpy(g.copy())
        opt.step()
        w, m, v = O.adamw(w, g, m, v, t, 1e-2, B1, B2, EPS, 0.03)
        assert np.allclose(w, p.detach().numpy(), rtol=1e-13, atol=0)


def test_oracle_codes_are_e4m3():
    ours = O.e4m3_values()
    theirs = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ours[~np.isnan(ours)], theirs[~np.isnan(theirs)])
    assert np.array_equal(np.isnan(ours), np.isnan(theirs))


def test_oracle_scale_is_the_smallest_that_fits():
    x = np.array([[0.0], [448.0], [np.nextafter(448.0, 1e3)], [1e-45], [FLT_MAX], [1.75], [1.76]]) * np.ones((1, 256))
    e = O.scale_bytes(x)
    assert list(e) == [1, 127, 128, 1, 247, 119, 120]
    for k in (1, 2, 4, 5, 6):
        assert x[k, 0] <= 448 * 2.0 ** (e[k] - 127) and x[k, 0] > 448 * 2.0 ** (e[k] - 128)


@pytest.mark.parametrize("square", [False, True])
def test_oracle_rounding_keeps_the_mean_and_the_codes(square):
    """Over all 65536 draws the mean of m, and of r^2, is the value's own to the draws' resolution, and a value that is
    a code already stays for every draw."""
    bits = np.arange(65536)
    codes = set(O.e4m3_values()[~np.isnan(O.e4m3_values())])
    e = np.array([127])
    for a in (300.3, 17.01, 0.02, 2.0 ** -6, 2.0 ** -6 * 0.999, 0.0007, 2.0 ** -9 * 0.25, 447.99):
        y, gap, _ = O.round_codes(np.full((1, 65536), a), e, bits, square)
        assert set(y.ravel()) <= codes
        want, got = (a * a, (y * y).mean()) if square else (a, y.mean())
        step = gap[0, 0] * (2 * y.min() + gap[0, 0] if square else 1.0)
        assert abs(got - want) <= step / 65536
    for a in (448.0, 0.0, 2.0 ** -9, 2.0 ** -6, 1.125, 30.0):
        y, _, _ = O.round_codes(np.full((1, 65536), a), e, bits, square)
        assert (y == a).all()


def test_oracle_random_bits_look_uniform():
    """Both halves of the 32 bits over 2^18 elements: 256 equal cells hold 1024 each, off by at most 6 standard
    deviations; neighbours, the halves, and one step and the next are uncorrelated (6 / sqrt(n))."""
    n = 1 << 18
    x = O.random_bits(1234567890123, 7, 0, n)
    y = O.random_bits(1234567890123, 8, 0, n)
    far = O.random_bits(1234567890123, 7, 1 << 32, n)
    halves = [(z & np.uint64(0xFFFF)).astype(float) for z in (x, y, far)] + [(x >> np.uint64(16)).astype(float)]
    for z in halves:
        cells = np.bincount((z // 256).astype(int), minlength=256)
        assert np.abs(cells - n / 256).max() <= 6 * math.sqrt(n / 256)
    lo, nxt, other, hi = halves
    for p, q in ((lo, nxt), (lo, other), (lo, hi), (lo[1:], lo[:-1]), (lo[256:], lo[:-256])):
        assert abs(np.corrcoef(p, q)[0, 1]) <= 6 / math.sqrt(n)


# --------------------------------------------------------------------------
# CPU: refusals, before anything reaches a device
# --------------------------------------------------------------------------
@pytest.fixture(scope="module")
def lib():
    from shampoo_second_order_b200 import build as B
    if not os.path.exists(L.LIB_PATH) or not os.path.exists(B.TENSORS):
        import __graft_entry__
        __graft_entry__.build()
    return L.lib()


@pytest.mark.parametrize("kw,msg", [
    (dict(numel=[]), "nparams"), (dict(numel=[4, 0]), "element count"), (dict(numel=[1 << 41]), "element count"),
    (dict(numel=[1 << 40] * 20), "more elements"),
    (dict(beta1=1.0), "beta1"), (dict(beta1=-0.1), "beta1"), (dict(beta2=1.0), "beta2"), (dict(beta2=float("nan")), "beta"),
    (dict(epsilon=0.0), "epsilon"), (dict(epsilon=1e-60), "epsilon"), (dict(epsilon=1e-39), "epsilon"), (dict(epsilon=float("inf")), "epsilon"),
    (dict(state_bits=16), "state_bits"), (dict(grad_dtype=7), "dtype"),
    (dict(max_norm=-1.0), "max_norm"), (dict(max_norm=float("nan")), "max_norm"),
    (dict(weight_decay=[-1.0]), "weight_decay"), (dict(weight_decay=[float("nan")]), "weight_decay"),
])
def test_adamw_create_refuses_bad_options(lib, kw, msg):
    args = dict(numel=[8], beta1=B1, beta2=B2, epsilon=EPS, weight_decay=[0.0], state_bits=32, grad_dtype=0, max_norm=0.0)
    args.update(kw)
    if "numel" in kw:
        args["weight_decay"] = [0.0] * len(kw["numel"])
    with pytest.raises(L.ShampooError) as e:
        L.shampoo_adamw_create(**args)
    assert e.value.status == L.EINVAL and msg in str(e.value)


@pytest.mark.parametrize("numel,dtype", [([], 0), ([0], 0), ([-3], 0), ([5], 2)])
def test_clip_create_refuses_bad_lists(lib, numel, dtype):
    with pytest.raises(L.ShampooError) as e:
        L.shampoo_clip_create(numel, dtype)
    assert e.value.status == L.EINVAL


def test_null_contexts_are_refused(lib):
    p = (C.c_void_p * 1)(16)
    n = C.c_int()
    assert lib.shampoo_clip_create(None, 1, (C.c_int64 * 1)(4), 0, None) == L.EINVAL
    assert lib.shampoo_clip_norm(None, p) == L.EINVAL
    assert lib.shampoo_clip_apply(None, p, 1.0) == L.EINVAL
    assert lib.shampoo_clip_result(None, p) == L.EINVAL
    assert lib.shampoo_clip_nonfinite_status(None, C.byref(n)) == L.EINVAL
    assert lib.shampoo_adamw_create(None, 1, (C.c_int64 * 1)(4), B1, B2, EPS, None, 32, 0, 0.0, 0, None) == L.EINVAL
    assert lib.shampoo_adamw_step(None, p, p, None, 0.1) == L.EINVAL
    assert lib.shampoo_adamw_state(None, 1, p, C.byref(C.c_int64())) == L.EINVAL
    assert lib.shampoo_adamw_offset(None, 0) == -1
    assert lib.shampoo_adamw_nonfinite_status(None, C.byref(n)) == L.EINVAL
    assert b"NULL" in lib.shampoo_adamw_last_error(None)
    assert lib.shampoo_clip_set_stream(None, None) == L.EINVAL
    assert lib.shampoo_adamw_set_stream(None, None) == L.EINVAL
    lib.shampoo_clip_destroy(None)
    lib.shampoo_adamw_destroy(None)


def test_lists_are_checked_before_the_library(lib):
    from array import array
    from shampoo_second_order_b200 import AdamW
    opt = object.__new__(AdamW)
    opt._numel, opt._device, opt.shapes = array("q", [6, 4]), 0, [(2, 3), (4,)]
    ok = [torch.zeros(2, 3), torch.zeros(4)]
    for bad, why in ((ok[:1], "expected 2"), ([torch.zeros(2, 3), torch.zeros(5)], "contiguous"), ([1, 2], "contiguous"),
                     ([torch.zeros(3, 2).t(), torch.zeros(4)], "contiguous"), ([None, ok[1]], "contiguous"),
                     ([torch.zeros(2, 3).bfloat16(), torch.zeros(4)], "contiguous"), (ok, "CUDA device 0")):
        with pytest.raises(ValueError, match=why):
            opt._pointers(bad, "grads", torch.float32)


@pytest.mark.gpu
def test_lists_of_the_wrong_tensors_are_refused(cuda):
    from shampoo_second_order_b200 import AdamW
    opt = AdamW([(2, 3), (4,)])
    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)   # noqa: E731
    g = [z(2, 3), z(4)]
    opt.step([z(6), torch.nn.Parameter(z(4))], tuple(g), 0.1)      # any shape of as many elements
    for bad in ([z(2, 3), z(5)], [z(3, 2).t(), z(4)], [z(2, 3), z(8)[::2]], [z(2, 3), z(4, dtype=torch.bfloat16)],
                [z(2, 3), z(4, dtype=torch.float16)], [z(2, 3), z(4, dtype=torch.int32)], [z(2, 3), torch.zeros(4)],
                [z(2, 3), torch.zeros(4, device="meta")], [z(2, 3), 4], [z(2, 3), z(2, 2).to_sparse()]):
        for lists in ((bad, g), (g, bad)):
            with pytest.raises(ValueError, match="contiguous"):
                opt.step(*lists, 0.1)
    with pytest.raises(ValueError, match="expected 2"):
        opt.step(g[:1], g, 0.1)
    with pytest.raises(ValueError, match="copies"):
        opt.step(g, g, 0.1, copies=g)


# --------------------------------------------------------------------------
# GPU
# --------------------------------------------------------------------------
gpu = pytest.mark.gpu


@pytest.fixture
def cuda(lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def f64(x):
    return x.detach().double().cpu().numpy().ravel()


class Params:
    """A list of float32 weights, gradients and bfloat16 copies, as a user holds them: `shift` None gives every
    tensor memory of its own, a number packs each list into one buffer without gaps from that element on, with
    guard elements at both ends."""

    def __init__(self, sizes, gdt, seed, shift=None, scale=1e-3):
        rng = np.random.default_rng(seed)
        self.sizes, self.gdt = sizes, torch.bfloat16 if gdt == "bf16" else torch.float32
        self.rng, self.scale, self.buffers = rng, scale, []
        self.w = self.place([rng.standard_normal(k) * 0.02 for k in sizes], torch.float32, shift)
        self.c = self.place([np.zeros(k) for k in sizes], torch.bfloat16, shift)
        self.g = self.place([self.draw(k) for k in sizes], self.gdt, shift)

    def draw(self, k):
        return self.rng.standard_normal(k) * self.scale * 10.0 ** self.rng.uniform(-2, 2)

    def place(self, xs, dtype, shift):
        if shift is None:
            return [torch.tensor(x, dtype=dtype, device="cuda") for x in xs]
        total = sum(len(x) for x in xs)
        buf = torch.full((shift + total + 8,), 7.0, dtype=dtype, device="cuda")
        out, at = [], shift
        for x in xs:
            out.append(buf[at:at + len(x)])
            out[-1].copy_(torch.tensor(x, dtype=dtype))
            at += len(x)
        self.buffers.append((buf, shift, at))
        return out

    def new_grads(self):
        for g, k in zip(self.g, self.sizes):
            g.copy_(torch.tensor(self.draw(k), dtype=self.gdt))

    def guards_intact(self):
        return all(bool((b[:s] == 7).all()) and bool((b[e:] == 7).all()) for b, s, e in self.buffers)


def moments(opt, i):
    """(m, v or r, their codes' rows' scale bytes) of parameter i in float64."""
    s, o, k = opt.state_tensors(), opt.offsets[i], opt._numel[i]
    if opt.state == "f32":
        return f64(s["m"][o:o + k]), f64(s["v"][o:o + k]), None
    blocks = slice(o // 256, (o + k + 255) // 256)
    val = O.e4m3_values()
    out, es = [], []
    for name in ("m", "r"):
        codes = s[name].view(torch.uint8)[o:o + -(-k // 256) * 256].cpu().numpy()
        e = s[name + "_scale"].view(torch.uint8)[blocks].cpu().numpy().astype(int)
        out.append((val[codes].reshape(-1, 256) * 2.0 ** (e[:, None] - 127.0)).ravel()[:k])
        es.append(e)
    return out[0], out[1], es


def check_codes(x, slop, got, got_e, bits, square):
    """The codes `got` of rows x (off by at most slop in 32 bits) with scale bytes got_e."""
    e = O.scale_bytes(x)
    rows = np.arange(len(e))
    edge = np.abs(np.abs(x).max(1) / (448.0 * 2.0 ** (np.minimum(e, got_e) - 127.0)) - 1.0)
    ok = (e == got_e) | (edge <= 40 * U)      # a largest magnitude on the border of two scales
    assert ok.all(), (rows[~ok], e[~ok], got_e[~ok])
    want, gap, slack = O.round_codes(x, got_e, bits, square)
    off = slop / (2.0 ** (got_e[:, None] - 127.0) * gap)
    # the lift by 2^-6 rounds once (2^-29 of gaps of 2^-9); r's probability takes eight more roundings of
    # terms up to 17 gaps, and moves by at most 17/8 for each gap that r moves
    off = 17.0 / 8.0 * off + 2.0 ** -20 + 8 * 17 * U if square else off + 2.0 ** -20
    wrong = (got != want) & (slack > off)
    assert not wrong.any(), (np.argwhere(wrong)[:5], got[wrong][:5], want[wrong][:5], slack[wrong][:5], off[wrong][:5])
    near = got != want
    assert (np.abs(np.abs(got) - np.abs(want))[near] <= 1.01 * gap[near]).all()


def check_step(opt, P, lr, decay, max_norm, seed, copies):
    """One opt.step() on P against the oracle started from the state and weights as they are."""
    n = len(P.sizes)
    before = [moments(opt, i) for i in range(n)]
    step0 = opt.state_tensors()["step"].cpu().numpy().copy()
    w0, g0, c0 = [f64(x) for x in P.w], [f64(x) for x in P.g], [f64(x) for x in P.c]
    opt.step(P.w, P.g, lr, copies=P.c if copies else None)
    torch.cuda.synchronize()
    norm, fine = O.global_norm(g0)
    assert abs(float(opt.grad_norm()) - norm) <= 10 * U * 1.01 * norm
    assert opt.nonfinite_status() == n - sum(fine)
    c = O.clip_factor(norm, max_norm)
    gerr = 10 if c != 1.0 else 0
    step1 = opt.state_tensors()["step"].cpu().numpy()
    for i in range(n):
        assert np.array_equal(f64(P.g[i]), g0[i], equal_nan=True)
        m1, v1, e1 = moments(opt, i)
        if not fine[i]:
            m0, v0, e0 = before[i]
            assert step1[i] == step0[i] and np.array_equal(m0, m1) and np.array_equal(v0, v1)
            assert np.array_equal(w0[i], f64(P.w[i])) and np.array_equal(c0[i], f64(P.c[i]))
            continue
        assert step1[i] == step0[i] + 1
        t = int(step1[i])
        m0, v0, _ = before[i]
        if opt.state == "8bit":
            v0 = v0 ** 2
        w, m, v = O.adamw(w0[i], c * g0[i], m0, v0, t, lr, B1, B2, EPS, decay[i])
        em = 1.01 * U * (2 * np.abs(B1 * m0) + (2 + gerr) * np.abs((1 - B1) * c * g0[i]) + np.abs(m)) + 1e-45
        ev = 1.01 * (6 + 2 * gerr) * U * v + 3e-45
        r = np.sqrt(v)
        first, d = lr / (1 - B1 ** t), r / math.sqrt(1 - B2 ** t) + EPS
        # where v is in the subnormal range r has an absolute error of sqrt(its)
        er = (5 + gerr) * U * r + np.where(v < 1e-37, 2e-22, 0.0)
        ew = 1.01 * (U * (np.abs(w0[i]) + np.abs(w)) + first / d * em
                     + first * np.abs(m) / d * (9 * U + er / math.sqrt(1 - B2 ** t) / d)) + 1e-45
        got = f64(P.w[i])
        assert (np.abs(got - w) <= ew).all(), (i, t, np.max(np.abs(got - w) / ew))
        if copies:   # the copy is this very weight, rounded to nearest
            assert torch.equal(P.c[i], P.w[i].bfloat16())
        if opt.state == "f32":
            assert (np.abs(m1 - m) <= em).all(), (i, np.max(np.abs(m1 - m) / em))
            assert (np.abs(v1 - v) <= ev).all(), (i, np.max(np.abs(v1 - v) / ev))
            continue
        k = len(m)
        bits = O.random_bits(seed, t, opt.offsets[i], -(-k // 256) * 256).reshape(-1, 256)
        for x, err, y, e, b, square in ((m, em, m1, e1[0], bits & np.uint64(0xFFFF), False),
                                        (r, er, v1, e1[1], bits >> np.uint64(16), True)):
            got = O.rows(y) / 2.0 ** (e[:, None] - 127.0)
            check_codes(O.rows(x), O.rows(err), got, e, b.astype(np.float64), square)
    if opt.state == "f32":
        used = np.zeros(opt.state_tensors()["m"].numel(), dtype=bool)
        for o, k in zip(opt.offsets, P.sizes):
            used[o:o + k] = True
        gap = torch.from_numpy(~used).cuda()
        assert not opt.state_tensors()["m"][gap].any() and not opt.state_tensors()["v"][gap].any()
    assert P.guards_intact()


SETS = {
    "one": [1],
    "tiny": [1, 2, 3, 5, 31],
    "block edges": [255, 256, 257, 4095, 511],
    "chunk edges": [8191, 8192, 8193, 16384 + 255],
    "mixed": [200 * 130, 64 * 64, 19 * 200, 130, 64, 77],
    "layer": [512 * 512, 512 * 1024, 512],
    "large edges": [8191, 8192, 8193, 1, 16384 + 255, 131072, 255, 50003],
}
# lists of up to 65536 elements take one launch, larger ones two: `more` brings a list over


@gpu
@pytest.mark.parametrize("state", ["f32", "8bit"])
@pytest.mark.parametrize("gdt", ["f32", "bf16"])
@pytest.mark.parametrize("name", list(SETS))
@pytest.mark.parametrize("shift", [None, 0, 1, 3])
def test_adamw_steps_match_the_oracle(cuda, state, gdt, name, shift):
    """Four steps from zero moments, with and without clipping and copies, at every alignment of the lists."""
    from shampoo_second_order_b200 import AdamW
    sizes = SETS[name]
    for clip, copies in ((False, False), (True, True)):
        P = Params(sizes, gdt, seed=11, shift=shift)
        decay = [0.1 * (i % 2) for i in range(len(sizes))]
        norm = math.sqrt(sum(float((f64(g) ** 2).sum()) for g in P.g))
        max_norm = 0.5 * norm if clip else 0.0
        opt = AdamW([(k,) for k in sizes], B1, B2, EPS, decay, state, gdt, max_norm, seed=-5)
        for t in range(4):
            check_step(opt, P, 10.0 ** -(1 + t), decay, max_norm, -5, copies)
            P.new_grads()


@gpu
@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_adamw_many_tensors(cuda, state):
    """More tensors than one launch's arguments hold (1024), and counts around the smaller argument blocks."""
    from shampoo_second_order_b200 import AdamW
    rng = np.random.default_rng(3)
    for n in (32, 33, 256, 257, 1024, 1025, 2100):
        sizes = [int(k) for k in rng.integers(1, 700, n)]
        P = Params(sizes, "f32", seed=n, shift=2)
        if n > 1024:
            P.g[1024][0] = float("nan")
        opt = AdamW([(k,) for k in sizes], B1, B2, EPS, 0.0, state, "f32", 1e-3, seed=9)
        for _ in range(2):
            check_step(opt, P, 1e-3, [0.0] * n, 1e-3, 9, False)


@gpu
@pytest.mark.parametrize("more", [[], [150000]])
@pytest.mark.parametrize("state", ["f32", "8bit"])
@pytest.mark.parametrize("gdt", ["f32", "bf16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_adamw_skips_gradients_that_are_not_finite(cuda, state, gdt, value, more):
    """At the first, the last and an inner element; then all of them; then none again: step counts differ from then on."""
    from shampoo_second_order_b200 import AdamW
    sizes = [9000, 300, 17, 8192] + more
    n = len(sizes)
    P = Params(sizes, gdt, seed=4)
    opt = AdamW([(k,) for k in sizes], B1, B2, EPS, 0.01, state, gdt, 1e-3, seed=1)
    check_step(opt, P, 1e-3, [0.01] * n, 1e-3, 1, True)
    for where in ((0, 0), (0, 8999), (1, 299), (2, 5), (3, 8191)):
        P.new_grads()
        P.g[where[0]][where[1]] = value
        check_step(opt, P, 1e-3, [0.01] * n, 1e-3, 1, True)
    for g in P.g:
        g[3] = value
    check_step(opt, P, 1e-3, [0.01] * n, 1e-3, 1, True)
    assert opt.nonfinite_status() == n and float(opt.grad_norm()) == 0.0
    P.new_grads()
    check_step(opt, P, 1e-3, [0.01] * n, 1e-3, 1, True)
    assert opt.state_tensors()["step"].tolist() == [5, 6, 6, 6] + [7] * len(more)


@gpu
@pytest.mark.parametrize("more", [[], [200000]])
@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_adamw_extreme_gradients(cuda, state, more):
    """Squares beyond and below the range of a float, zeros, and the largest float: finite results, a norm, and beyond
    2^63 the step of a gradient of 2^63."""
    from shampoo_second_order_b200 import AdamW
    for value in (1e25, 3.4028234663852886e38, 1e-25, 1e-38, 0.0):
        sizes = [1000, 300] + more
        P = Params(sizes, "f32", seed=6)
        for g in P.g:
            g.copy_(torch.sign(g) * value)
        opt = AdamW([(k,) for k in sizes], B1, B2, EPS, 0.0, state, "f32")
        w0 = [f64(w) for w in P.w]
        for t in range(3):
            opt.step(P.w, P.g, 1e-2)
            norm = value * math.sqrt(sum(sizes))
            assert float(opt.grad_norm()) == pytest.approx(norm if norm < FLT_MAX else math.inf, rel=1e-6)
        for i, w in enumerate(P.w):
            assert np.isfinite(f64(w)).all() and np.isfinite(moments(opt, i)[0]).all() and np.isfinite(moments(opt, i)[1]).all()
            if value == 0.0:
                assert np.array_equal(f64(w), w0[i])
            if value > 2.0 ** 63 and state == "f32":
                g = np.sign(f64(P.g[i])) * 2.0 ** 63
                m, v = g * (1 - B1 ** 3), g * g * (1 - B2 ** 3)
                assert (np.abs(moments(opt, i)[0] - m) <= 12 * U * np.abs(m)).all()
                assert (np.abs(moments(opt, i)[1] - v) <= 18 * U * v).all()


@gpu
def test_adamw_clips_gradients_beyond_the_range_of_their_squares(cuda):
    from shampoo_second_order_b200 import AdamW
    P = Params([5000, 100], "f32", seed=8)
    for g in P.g:
        g.mul_(1e24)
    opt = AdamW([(5000,), (100,)], B1, B2, EPS, 0.0, "f32", "f32", max_norm=1.0)
    check_step(opt, P, 1e-3, [0.0, 0.0], 1.0, 0, False)


def codes_of_f32(x, bits, square):
    """(e4m3 values, scale bytes) of float32 rows x >= 0 or of any sign, each operation rounded to float32."""
    e = (((x.abs().amax(1).view(torch.int32) + 0x1FFFFF) >> 23) - 8).clamp(min=1)
    a = torch.ldexp(x.abs(), (127 - e)[:, None])
    lift = torch.where(a < 2.0 ** -6, 2.0 ** -6, 0.0)
    word = (a + lift).view(torch.int32)
    if square:
        lo = (word & -0x100000).view(torch.float32) - lift
        gap = (word & 0x7F800000).view(torch.float32) * 0.125
        y = torch.where((a - lo) * (a + lo) > bits.float() * 2.0 ** -16 * (gap * (2.0 * lo + gap)), lo + gap, lo)
    else:
        y = ((word + (bits.int() << 4)) & -0x100000).view(torch.float32) - lift
    return torch.copysign(y, x), e


@gpu
@pytest.mark.parametrize("gdt", ["f32", "bf16"])
@pytest.mark.parametrize("n,shift", [(1 << 22, 0), (1 << 20, 1), (1 << 20, 2), (5000001, 2), (40000, 0), (40000, 3)])
def test_8bit_codes_are_those_of_operations_rounded_one_by_one(cuda, gdt, n, shift):
    """Every code equal, with no tolerance: a product fused with its sum changes a last bit in a fifth of the moments, and
    the code of about one element in a million; two steps on, at both alignments and in both kernels."""
    from shampoo_second_order_b200 import AdamW
    gen = torch.Generator("cuda").manual_seed(n + shift)
    size = torch.exp(2.0 * torch.randn(n, device="cuda", generator=gen)) * 1e-3
    opt = AdamW([(n,)], B1, B2, EPS, 0.0, "8bit", gdt, seed=12)
    w = torch.zeros(n + shift, device="cuda")[shift:]
    b1, omb1, b2, omb2 = (torch.tensor(x, dtype=torch.float32, device="cuda") for x in (B1, 1 - B1, B2, 1 - B2))
    for t in (1, 2, 3):
        g = torch.empty(n + shift, device="cuda", dtype=torch.bfloat16 if gdt == "bf16" else torch.float32)[shift:]
        g.copy_(torch.randn(n, device="cuda", generator=gen) * size)
        s = {k: x.clone() for k, x in opt.state_tensors().items()}
        opt.step([w], [g], 1e-3)
        pad = -n % 256
        x = torch.nn.functional.pad(g.float(), (0, pad)).view(-1, 256)
        m0 = s["m"].float().view(-1, 256) * s["m_scale"].float()[:, None]
        r0 = s["r"].float().view(-1, 256) * s["r_scale"].float()[:, None]
        m = b1 * m0 + omb1 * x
        r = (b2 * (r0 * r0) + omb2 * x * x).sqrt()
        bits = torch.from_numpy(O.random_bits(12, t, 0, n + pad).astype(np.int64)).cuda().view(-1, 256)
        now = opt.state_tensors()
        for name, y, b, square in (("m", m, bits & 0xFFFF, False), ("r", r, bits >> 16, True)):
            want, e = codes_of_f32(y, b, square)
            assert torch.equal(now[name + "_scale"].view(torch.uint8).int(), e)
            got = now[name].float().view(-1, 256)
            assert torch.equal(got, want), ((got != want).sum(), (got != want).nonzero()[:4])


@gpu
def test_8bit_moments_have_no_drift(cuda):
    """Two thousand steps on noise: the mean of v over 2^16 elements follows the one in 32 bits.  The stochastic
    rounding is unbiased; its noise is about 0.3 v an element once the moments have settled, 0.3 / 256 of the mean: 2 %
    is some fifteen standard deviations.  Rounding to nearest, or r by its own fraction, is further off than that.
    m likewise: its mean square exceeds the 32-bit one by the rounding's variance, at most a few percent."""
    from shampoo_second_order_b200 import AdamW
    n = 1 << 16
    gen = torch.Generator("cuda").manual_seed(5)
    a, b = (AdamW([(n,)], B1, B2, EPS, 0.0, s, "f32", seed=77) for s in ("f32", "8bit"))
    w = [torch.zeros(n, device="cuda") for _ in range(2)]
    size = torch.exp(torch.randn(n, device="cuda", generator=gen))   # gradients of different sizes within a block
    for _ in range(2000):
        g = torch.randn(n, device="cuda", generator=gen) * size
        a.step([w[0]], [g], 1e-4)
        b.step([w[1]], [g], 1e-4)
    v, (_, r, _) = moments(a, 0)[1], moments(b, 0)
    s2 = f64(size) ** 2
    assert abs((r * r / s2).mean() / (v / s2).mean() - 1.0) <= 0.02
    assert abs(np.log(r * r / v)).max() <= math.log(30.0)   # and no element is stuck


@gpu
@pytest.mark.parametrize("gdt", ["f32", "bf16"])
@pytest.mark.parametrize("name", list(SETS))
@pytest.mark.parametrize("shift", [None, 1, 2])
def test_clip_matches_the_oracle(cuda, gdt, name, shift):
    from shampoo_second_order_b200 import GradClip
    sizes = SETS[name]
    P = Params(sizes, gdt, seed=21, shift=shift)
    op = GradClip([(k,) for k in sizes], gdt)
    for factor in (0.3, 1.5, 0.999):
        g0 = [f64(g) for g in P.g]
        norm, _ = O.global_norm(g0)
        assert abs(float(op.norm(P.g)) - norm) <= 10 * U * 1.01 * norm
        assert all(np.array_equal(f64(g), x) for g, x in zip(P.g, g0))
        got = op.clip(P.g, factor * norm)
        assert abs(float(got) - norm) <= 10 * U * 1.01 * norm and op.nonfinite_status() == 0
        c = O.clip_factor(norm, factor * norm)
        for g, x in zip(P.g, g0):
            if c == 1.0:
                assert np.array_equal(f64(g), x)
            else:
                half = 2.0 ** -8 if gdt == "bf16" else U
                assert (np.abs(f64(g) - c * x) <= 1.01 * (10 * U + half) * np.abs(c * x) + 1e-40).all()
        assert P.guards_intact()


@gpu
@pytest.mark.parametrize("more", [0, 150000])
def test_clip_leaves_out_what_is_not_finite(cuda, more):
    from shampoo_second_order_b200 import GradClip
    sizes = [10000 + more, 77, 256]
    P = Params(sizes, "f32", seed=22)
    P.g[1][76] = float("inf")
    g0 = [f64(g) for g in P.g]
    op = GradClip([(k,) for k in sizes])
    norm = math.sqrt((g0[0] ** 2).sum() + (g0[2] ** 2).sum())
    assert float(op.clip(P.g, norm / 4)) == pytest.approx(norm, rel=10 * U)
    assert op.nonfinite_status() == 1 and np.array_equal(f64(P.g[1]), g0[1])
    for i in (0, 2):
        assert (np.abs(f64(P.g[i]) - g0[i] / 4) <= 12 * U * np.abs(g0[i]) / 4).all()


@gpu
@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_same_inputs_give_the_same_bits(cuda, state):
    from shampoo_second_order_b200 import AdamW
    sizes = [100000, 33, 70001]
    out = []
    for _ in range(2):
        P = Params(sizes, "f32", seed=31)
        opt = AdamW([(k,) for k in sizes], state=state, max_norm=1e-2, seed=4)
        for _ in range(3):
            opt.step(P.w, P.g, 1e-3)
        out.append([w.clone() for w in P.w] + [x.view(torch.uint8).clone() for x in opt.state_tensors().values()])
    assert all(torch.equal(x, y) for x, y in zip(*out))


@gpu
@pytest.mark.parametrize("more", [[], [150000]])
@pytest.mark.parametrize("own_stream", [False, True])
@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_adamw_in_a_graph_and_on_other_streams(cuda, state, own_stream, more):
    """A captured step replayed, eager steps between the replays with other tensors, a second graph of the same
    context, and steps from other streams, with and without a stream of the context's own: all give what eager
    steps on one stream give."""
    from shampoo_second_order_b200 import AdamW
    sizes = [5000, 256, 3] + more
    make = lambda: (Params(sizes, "bf16", seed=41), Params(sizes, "bf16", seed=42),   # noqa: E731
                    AdamW([(k,) for k in sizes], state=state, grad_dtype="bf16", max_norm=1e-2, seed=6))
    P, Q, ref = make()
    for X in (P, P, Q, P, Q, Q):
        ref.step(X.w, X.g, 1e-3, copies=X.c)
    want = P.w + Q.w + P.c + list(ref.state_tensors().values())
    A, B, opt = make()
    if own_stream:
        opt = AdamW([(k,) for k in sizes], state=state, grad_dtype="bf16", max_norm=1e-2, seed=6, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    graphs = []
    for X in (A, B):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):      # on a stream of torch's own
            opt.step(X.w, X.g, 1e-3, copies=X.c)
        graphs.append(graph)
    side = torch.cuda.Stream()
    graphs[0].replay()
    opt.step(A.w, A.g, 1e-3, copies=A.c)
    graphs[1].replay()
    graphs[0].replay()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        opt.step(B.w, B.g, 1e-3, copies=B.c)
    torch.cuda.current_stream().wait_stream(side)
    opt.step(B.w, B.g, 1e-3, copies=B.c)
    torch.cuda.synchronize()
    got = A.w + B.w + A.c + list(opt.state_tensors().values())
    for x, y in zip(want, got):
        assert torch.equal(x.view(torch.uint8) if x.element_size() == 1 else x, y.view(torch.uint8) if y.element_size() == 1 else y)


@gpu
def test_many_contexts_at_once(cuda):
    """Sixteen contexts of one to 1500 tensors, eager and as graphs, on five streams at a time: each ends where it ends
    when it runs alone."""
    import random
    from shampoo_second_order_b200 import AdamW

    def make(seed):
        r = random.Random(seed)
        n, total = r.choice([1, 3, 40, 300, 1500]), r.choice([500, 60000, 70000, 900000, 3000000])
        sizes = [max(1, int(total / n * r.uniform(0.2, 2.0))) for _ in range(n)]
        gdt, state = r.choice(["f32", "bf16"]), r.choice(["f32", "8bit"])
        gen = torch.Generator("cuda").manual_seed(seed)
        w = torch.randn(sum(sizes), device="cuda", generator=gen) * 0.02
        g = (torch.randn(sum(sizes), device="cuda", generator=gen) * 1e-3).to(torch.bfloat16 if gdt == "bf16" else torch.float32)
        b = torch.zeros(sum(sizes), device="cuda", dtype=torch.bfloat16)
        opt = AdamW([(k,) for k in sizes], state=state, grad_dtype=gdt, max_norm=r.choice([0, 0.1]), seed=seed)
        lists = [list(torch.split(x, sizes)) for x in (w, g, b)]
        return opt, lambda: opt.step(lists[0], lists[1], 1e-3, copies=lists[2]), w, b

    def ends(opt, step, w, b):
        return [x.view(torch.uint8).clone() for x in (w, b, *opt.state_tensors().values())]

    want = []
    for seed in range(16):
        alone = make(seed)
        for _ in range(5):
            alone[1]()
        want.append(ends(*alone))
    runs, calls = [make(seed) for seed in range(16)], []
    torch.cuda.synchronize()
    for seed, run in enumerate(runs):
        if seed % 3:
            calls.append(run[1])
            continue
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run[1]()
        calls.append(graph.replay)
    streams, rnd = [torch.cuda.Stream() for _ in range(5)], random.Random(0)
    torch.cuda.synchronize()
    for _ in range(5):
        for seed in rnd.sample(range(16), 16):
            with torch.cuda.stream(streams[seed % 5]):
                calls[seed]()
    torch.cuda.synchronize()
    for seed, run in enumerate(runs):
        assert all(torch.equal(x, y) for x, y in zip(want[seed], ends(*run))), seed


@gpu
def test_adamw_refuses_lists_that_overlap(cuda):
    from shampoo_second_order_b200 import AdamW, GradClip
    buf, g = torch.zeros(100, device="cuda"), torch.zeros(2, 40, device="cuda")
    opt = AdamW([(40,), (40,)])
    half = torch.zeros(2, 40, device="cuda", dtype=torch.bfloat16)
    for params, grads, copies in (([buf[:40], buf[:40]], list(g), None), ([buf[40:80], buf[1:41]], list(g), None),
                                  ([buf[:40], buf[40:80]], [g[0], buf[60:100]], None),
                                  ([buf[:40], buf[40:80]], list(g), [half[0], half[0]])):
        with pytest.raises(L.ShampooError, match="overlaps") as e:
            opt.step(params, grads, 0.1, copies=copies)
        assert e.value.status == L.EINVAL
    opt.step([buf[40:80], buf[:40]], [g[0], g[0]], 0.1)      # the same gradient twice is only read
    op = GradClip([(40,), (40,)])
    op.norm([g[0], g[0]])
    with pytest.raises(L.ShampooError, match="overlaps"):
        op.clip([g[0], g[0]], 1.0)
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(L.ShampooError, match="max_norm"):
            op.clip(list(g), bad)
    for lr in (-1.0, float("nan"), float("inf")):
        with pytest.raises(L.ShampooError, match="lr"):
            opt.step([buf[:40], buf[40:80]], list(g), lr)
    with pytest.raises(ValueError, match="weight_decay"):
        AdamW([(4,), (5,)], weight_decay=[0.1])
    with pytest.raises(ValueError, match="state"):
        AdamW([(4,)], state="16bit")
    p = (C.c_void_p * 2)(buf.data_ptr() + 2, buf.data_ptr() + 200)
    q = (C.c_void_p * 2)(g.data_ptr(), g.data_ptr() + 160)
    with pytest.raises(L.ShampooError, match="aligned"):
        L.shampoo_adamw_step(opt._ctx, p, q, None, 0.1)
    with pytest.raises(L.ShampooError, match="NULL"):
        L.shampoo_adamw_step(opt._ctx, (C.c_void_p * 2)(buf.data_ptr(), 0), q, None, 0.1)
    opt.close()
    with pytest.raises(RuntimeError, match="closed"):
        opt.step([buf[:40], buf[40:80]], list(g), 0.1)


@gpu
@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_adamw_state_is_saved_and_restored(cuda, state):
    from shampoo_second_order_b200 import AdamW
    sizes = [3000, 11]
    P = Params(sizes, "f32", seed=51)
    opt = AdamW([(k,) for k in sizes], state=state, seed=2)
    for _ in range(3):
        opt.step(P.w, P.g, 1e-3)
    saved = {k: x.clone() for k, x in opt.state_tensors().items()}
    view, w = opt.state_tensors()["step"], [x.clone() for x in P.w]
    opt.step(P.w, P.g, 1e-3)
    want = [x.clone() for x in P.w]
    opt.close()
    del opt
    assert view.tolist() == [4, 4]      # a view keeps the memory it views
    again = AdamW([(k,) for k in sizes], state=state, seed=2)
    for k, x in again.state_tensors().items():
        x.view(torch.uint8).copy_(saved[k].view(torch.uint8))
    again.step(w, P.g, 1e-3)
    assert all(torch.equal(x, y) for x, y in zip(w, want))


@gpu
@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_adamw_beyond_32_bit_offsets(cuda, state):
    """Two tensors, the first of 5000 elements more than 2^31, or 2^32 with 8-bit moments: what lies behind that in the first,
    and the second, whose moments begin there, step as the oracle says; the clipping reaches them too."""
    from shampoo_second_order_b200 import AdamW, GradClip
    n, tail, small = (1 << (31 if state == "f32" else 32)) + 5000, 20000, 700
    if torch.cuda.mem_get_info()[0] < 50 << 30:
        pytest.skip("needs 50 GB of device memory")
    gen = torch.Generator("cuda").manual_seed(1)
    w, w2 = torch.zeros(n, device="cuda"), torch.randn(small, device="cuda", generator=gen) * 0.02
    g, g2 = torch.zeros(n, device="cuda", dtype=torch.bfloat16), (torch.randn(small, device="cuda", generator=gen) * 1e-3).bfloat16()
    x = torch.randn(tail, device="cuda", generator=gen)
    w[-tail:] = x * 0.02
    g[-tail:] = (x.flip(0) * 1e-3).bfloat16()
    opt = AdamW([(n,), (small,)], B1, B2, EPS, 0.1, state, "bf16", seed=3)
    assert opt.offsets == [0, (n + 255) // 256 * 256]
    cases = [(f64(w[-tail:]), f64(g[-tail:]), w[-tail:], n - tail), (f64(w2), f64(g2), w2, opt.offsets[1])]
    opt.step([w, w2], [g, g2], 1e-2)
    norm, _ = O.global_norm([f64(g[-tail:]), f64(g2)])
    assert abs(float(opt.grad_norm()) - norm) <= 10 * U * 1.01 * norm
    assert not w[:-tail].any()
    s = opt.state_tensors()
    for w0, g0, now, first in cases:
        want, m, v = O.adamw(w0, g0, np.zeros(len(w0)), np.zeros(len(w0)), 1, 1e-2, B1, B2, EPS, 0.1)
        assert (np.abs(f64(now) - want) <= 40 * U * (np.abs(w0) + 1e-2)).all()
        at = -(-first // 256) * 256          # whole blocks from here on
        k = (len(m) - (at - first)) // 256 * 256
        m, v = m[at - first:][:k], v[at - first:][:k]
        if state == "f32":
            assert (np.abs(f64(s["m"][at:at + k]) - m) <= 6 * U * np.abs(m)).all()
            assert (np.abs(f64(s["v"][at:at + k]) - v) <= 6 * U * v).all()
            continue
        for name, x, square in (("m", m, False), ("r", np.sqrt(v), True)):
            e = s[name + "_scale"].view(torch.uint8)[at // 256:(at + k) // 256].cpu().numpy().astype(int)
            codes = O.e4m3_values()[s[name].view(torch.uint8)[at:at + k].cpu().numpy()].reshape(-1, 256)
            bits = O.random_bits(3, 1, at, k).reshape(-1, 256)
            bits = (bits >> np.uint64(16) if square else bits & np.uint64(0xFFFF)).astype(np.float64)
            check_codes(O.rows(x), 30 * U * np.abs(O.rows(x)), codes, e, bits, square)
    del opt, s, w
    torch.cuda.empty_cache()
    clip = GradClip([(n,), (small,)], "bf16")
    assert abs(float(clip.clip([g, g2], norm / 2)) - norm) <= 10 * U * 1.01 * norm
    for now, was in ((g[-tail:], cases[0][1]), (g2, cases[1][1])):
        assert (np.abs(f64(now) - was / 2) <= 1.01 * (10 * U + 2.0 ** -8) * np.abs(was) / 2).all()


@gpu
@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_shampoo_and_adamw_share_a_clipped_step(cuda, state):
    """As they are used together: all gradients are clipped to one norm, Shampoo steps the matrices, AdamW the
    embedding and the vectors, against both oracles."""
    from oracle import ShampooOracle
    from shampoo_second_order_b200 import AdamW, GradClip, Shampoo, workloads as wl
    mats, rest = [(100, 64), (64, 130)], [(500, 24), (64,), (130,)]
    shapes = mats + rest
    W = [torch.from_numpy(w).cuda() for w in wl.make_params(shapes, 61)]
    Wo = [f64(w).reshape(s) for w, s in zip(W, shapes)]
    clip = GradClip(shapes)
    sh = Shampoo(mats, 64, 0.99, 1e-6)
    ad = AdamW(rest, B1, B2, EPS, 0.01, state, "f32", seed=8)
    oracle = ShampooOracle(mats, 64, 0.99, 1e-6, 4, 1, 0.0)
    lr = 0.01
    for t in range(3):
        g = wl.make_grads(shapes, 61, t, 1e-2)
        G = [torch.from_numpy(x).cuda() for x in g]
        norm, _ = O.global_norm([x.astype(np.float64) for x in g])
        clip.clip(G, norm / 3)
        ad_before = [moments(ad, i) for i in range(3)]
        w_before = [f64(w) for w in W]
        sh.step(W[:2], G[:2], lr, True)
        ad.step(W[2:], G[2:], lr)
        torch.cuda.synchronize()
        prev = Wo[:2]
        Wo[:2] = oracle.step(prev, [x.astype(np.float64) / 3 for x in g[:2]], lr, True)
        for i in range(2):
            d, ref = f64(W[i]) - w_before[i], (Wo[i] - prev[i]).ravel()
            assert np.linalg.norm(d - ref) <= 1e-3 * np.linalg.norm(ref)      # the Shampoo step's own bound
        for i in range(3):
            m0, v0, _ = ad_before[i]
            v0 = v0 ** 2 if state == "8bit" else v0
            want, _, _ = O.adamw(w_before[2 + i], g[2 + i].astype(np.float64).ravel() / 3, m0, v0, t + 1, lr, B1, B2, EPS, 0.01)
            assert (np.abs(f64(W[2 + i]) - want) <= 1.01 * (2 * U * np.abs(want) + 100 * U * lr * 3.2)).all()
    sh.close()


@gpu
@pytest.mark.parametrize("args,says", [(["--optimizer", "adamw"], "adamw"), (["--optimizer", "adamw8", "--max-norm", "0.5"], "adamw8"),
                                       (["--max-norm", "0.5"], "pair tiles")])
def test_run_steps_command(cuda, capsys, args, says):
    from shampoo_second_order_b200 import run_steps
    assert run_steps.main(["--config", "transformer_layer_b512", "--params", "2", "--steps", "2"] + args) == 0
    assert f"({says})" in capsys.readouterr().out
