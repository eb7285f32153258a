"""GPU tests of the expert operators where a call is easily answered wrongly: rows that no expert holds, scores whose
parts cancel or leave the fp32 range, tails of an activation, router rows that are not finite, offsets that fall, and
sizes near what a launch can hold.  The plain fp64 references and their bounds are those of experts_reference.py."""
import math

import pytest

torch = pytest.importorskip("torch")

import experts_reference as ref  # noqa: E402
import test_gpu_experts as base  # noqa: E402

import differentiable_soft_top_amd as stk  # noqa: E402

pytestmark = pytest.mark.gpu

gen, within = base.gen, base.within


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no ROCm device")
    return torch.device("cuda:0")


# ---- the residual's gradient behind the last row -----------------------------

RESIDUALS = [p for p in base.PRODUCTS if p[8] and p[10] > 0.0]


def residual_gradient(dy, offsets):
    """y_r = act(z_r) + residual_r before offsets[E], 0 behind: dy there, 0 behind."""
    want = dy.clone()
    want[int(offsets[-1]):] = 0
    return want


@pytest.mark.parametrize("T,k,E,K,N,act,dtype,bias,residual,gather,dropped", RESIDUALS)
@pytest.mark.parametrize("odd", [False, True])
def test_product_residual_with_dropped_pairs(dev, T, k, E, K, N, act, dtype, bias, residual, gather, dropped, odd):
    print("[residual] T=%d K=%d N=%d odd=%d" % (T, K, N, odd), flush=True)
    x, w, offsets, rows, slots, b, res, dy = base.product_inputs(T, k, E, K, N, act, dtype, bias, residual, gather,
                                                                 dropped)
    total = int(offsets[-1])
    assert total < T * k
    dy[total:] = math.nan  # reaches nothing
    plan = stk.Dispatch(*(None if t is None else t.to(dev) for t in (offsets, rows, slots)))
    leaves = [base.place(t, dev, odd) for t in (x, w, b, res)]
    leaves = [None if t is None else t.requires_grad_(True) for t in leaves]
    y = stk.experts_product(leaves[0], leaves[1], plan, bias=leaves[2], act=act, residual=leaves[3])
    given = [t for t in leaves if t is not None]
    grads = torch.autograd.grad(y, given, base.place(dy, dev, odd))
    want = ref.product(x, w, offsets, rows, b, act, res, dy)
    for got, (value, bound), what in zip((y,) + grads, want, ("y", "dx", "dw", "db")[:len(given)]):
        within(got, value, bound, what)
    assert torch.equal(grads[-1].cpu(), residual_gradient(dy, offsets))
    assert torch.equal(stk.experts_residual_backward(base.place(dy, dev, odd), plan), grads[-1])


def test_product_residual_by_differences(dev):
    # moving the residual behind the last row moves nothing
    x, w, offsets, rows, slots, b, res, dy = base.product_inputs(40, 2, 5, 64, 24, "silu", "bf16", True, True, True, 0.4)
    plan = stk.Dispatch(offsets.to(dev), rows.to(dev), slots.to(dev))
    total = int(offsets[-1])
    leaf = res.to(dev).requires_grad_(True)

    def loss(r):
        y = stk.experts_product(x.to(dev), w.to(dev), plan, bias=b.to(dev), act="silu", residual=r)
        return (y.double() * dy.to(dev).double()).sum()

    with torch.no_grad():
        moved = leaf.clone()
        moved[total:] += 1
        assert float(loss(moved)) == float(loss(leaf))
    (grad,) = torch.autograd.grad(loss(leaf), [leaf])
    assert torch.equal(grad.cpu(), residual_gradient(dy, offsets))


@pytest.mark.parametrize("kept", [0, 1, 333])
def test_residual_gradient_of_none_and_all_rows(dev, kept):
    # alone (x, w and bias need no gradient), from a sum: a gradient without storage of its own
    N = 37
    offsets = torch.tensor([0, 0, kept], dtype=torch.int32)
    x, w = torch.randn(333, 16, generator=gen(1)).half(), torch.randn(2, N, 16, generator=gen(2)).half()
    res = torch.zeros(333, N, dtype=torch.float16, device=dev, requires_grad=True)
    y = stk.experts_product(x.to(dev), w.to(dev), stk.Dispatch(offsets.to(dev)), residual=res)
    (grad,) = torch.autograd.grad(y.sum(), [res])
    want = torch.zeros(333, N, dtype=torch.float16)
    want[:kept] = 1
    assert torch.equal(grad.cpu(), want)


def test_residual_gradient_behind_4_gib(dev):
    P, N = 1_100_000, 2048
    kept = P - 3
    dy = torch.ones(P, N, dtype=torch.bfloat16, device=dev)
    plan = stk.Dispatch(torch.tensor([0, 5, kept], dtype=torch.int32, device=dev))
    grad = stk.experts_residual_backward(dy, plan)
    assert (grad[kept:] == 0).all() and (grad[:kept] == 1).all()


def test_residual_gradient_captured_and_replayed(dev):
    dy = torch.randn(500, 72, generator=gen(3)).to(torch.bfloat16).to(dev)
    offsets = torch.tensor([0, 100, 500], dtype=torch.int32, device=dev)
    plan = stk.Dispatch(offsets)
    stk.experts_residual_backward(dy, plan)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = stk.experts_residual_backward(dy, plan)
    for kept in (500, 0, 123, 499):
        offsets[2] = kept
        want = stk.experts_residual_backward(dy, plan)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(out.cpu(), residual_gradient(dy.cpu(), [kept]))


# ---- softmax over the whole row ------------------------------------------------

WHOLE = [(3, 2, 1, "f32"), (70, 60, 4, "f32"), (33, 256, 8, "bf16"), (9, 500, 16, "f16"), (5, 1024, 32, "f32")]


@pytest.mark.parametrize("T,E,k,dtype", WHOLE)
@pytest.mark.parametrize("grouped", [False, True])
def test_softmax_weights_are_rounded_once(dev, T, E, k, dtype, grouped):
    z = (torch.randn(T, E, generator=gen(E)) * 4).to(base.DTYPES[dtype])
    options = dict(renormalize=False)
    if grouped:
        options.update(n_group=2, topk_group=2)
    w, e = stk.route(z.to(dev), k, **options)
    want_w, want_e = ref.route(z, k, **options)
    assert torch.equal(e.cpu(), want_e)
    within(w, want_w, want_w * 1.01 * ref.U32 + 1e-40, "weights")


@pytest.mark.parametrize("E", [1, 4, 16, 31])
def test_softmax_gradient_of_the_whole_sum_is_none(dev, E):
    # all chosen and equal cotangents: sum p = 1, so the gradient is 0; what is left are some E + 8 fp64 roundings of p
    z = torch.randn(40, E, generator=gen(E)) * 3
    zd = z.to(dev).requires_grad_(True)
    w, _ = stk.route(zd, E, renormalize=False)
    (dz,) = torch.autograd.grad(w, [zd], torch.full((40, E), 0.75, device=dev))
    p = torch.softmax(z.double(), 1)
    within(dz, torch.zeros(40, E, dtype=torch.float64), p * 0.75 * (E + 8) * 2.0 ** -52 + 1e-40, "dz")


@pytest.mark.parametrize("E,k,dtype", [(64, 4, "f32"), (256, 8, "f32"), (300, 12, "f16"), (1000, 20, "bf16")])
def test_softmax_gradient_where_the_chosen_hold_nearly_all(dev, E, k, dtype):
    # dz = p (g - sum g p) with equal g: p g (1 - sum of the chosen p), some 1e-7 of p g; a sum and a p that agree to
    # 2^-52 leave (E + 8) 2^-52 p g beside the rounding of the result
    z = torch.randn(20, E, generator=gen(k)) * 0.5 - 18
    for t in range(20):
        z[t, torch.randperm(E, generator=gen(t))[:k]] += 18
    z = z.to(base.DTYPES[dtype])
    zd = z.to(dev).requires_grad_(True)
    w, e = stk.route(zd, k, renormalize=False)
    g = torch.full((20, k), 1.25)
    (dz,) = torch.autograd.grad(w, [zd], g.to(dev))
    want = ref.route_grad(z, e.cpu(), g, renormalize=False)
    p = torch.softmax(z.double(), 1)
    within(dz, want, want.abs() * (1.01 * ref.half_step(z.dtype) + 2.0 ** -22) + p * 1.25 * (E + 8) * 2.0 ** -52
           + ref.tiny(z.dtype), "dz")


# ---- tails of the activations ---------------------------------------------------

def tail(dtype):
    z = -torch.arange(1, 401).double() / 32  # to -12.5, where z Phi(z) is 5e-35
    return z.to(base.DTYPES[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gelu_keeps_its_negative_tail(dev, dtype):
    # x = z, w = 1: z itself.  Phi(z) = erfc(-z / sqrt 2) / 2, whose argument is off by 2 2^-24 of itself: (z^2 + 2)
    # 2^-23 of the value; erfc by some 16 2^-24; the product and the rounding of y
    x = tail(dtype)[:, None]
    w = torch.ones(1, 1, 1, dtype=x.dtype)
    offsets = torch.tensor([0, len(x)], dtype=torch.int32)
    xd = x.to(dev).requires_grad_(True)
    y = stk.experts_product(xd, w.to(dev), stk.Dispatch(offsets.to(dev)), act="gelu")
    z = x.double()
    cdf = torch.special.erfc(-z / math.sqrt(2.0)) / 2
    value = z * cdf
    rel = (32 + 2 * z * z) * ref.U32
    within(y, value, value.abs() * (rel + 1.01 * ref.half_step(x.dtype)) + ref.tiny(x.dtype), "y")
    # the slope Phi(z) + z phi(z): the exponential's argument is off by some 4 2^-24 of itself
    (dx,) = torch.autograd.grad(y, [xd], torch.ones_like(y))
    bell = z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    slope = cdf + bell
    bound = (cdf + bell.abs()) * (32 + 4 * z * z) * ref.U32
    within(dx, slope, bound + slope.abs() * 1.01 * ref.half_step(x.dtype) + ref.tiny(x.dtype), "dx")


# ---- router rows that are not finite ---------------------------------------------

@pytest.mark.parametrize("score", ["softmax", "sigmoid", "given"])
@pytest.mark.parametrize("with_residual", [False, True])
def test_layer_shows_a_router_row_that_is_not_finite(dev, score, with_residual):
    # tokens 3 and 70 have a broken row of scores, token 5 is padding
    x, scores, w_up, w_down = base.layer_inputs()
    padded = scores.clone()
    padded[[3, 5, 70]] = -math.inf
    scores[5] = -math.inf
    scores[3, 7] = math.nan
    scores[70, 0] = math.inf
    leaves = [t.to(dev).requires_grad_(True) for t in (x, scores, w_up, w_down)]
    residual = leaves[0] if with_residual else None
    out, experts = stk.moe(*leaves, 3, residual=residual, score=score)
    want, _ = stk.moe(x.to(dev), padded.to(dev), w_up.to(dev), w_down.to(dev), 3,
                      residual=x.to(dev) if with_residual else None, score=score)
    broken = torch.zeros(x.shape[0], dtype=torch.bool, device=dev)
    broken[[3, 70]] = True
    assert (experts[[3, 5, 70]] == -1).all()
    assert torch.isnan(out[broken]).all()
    assert torch.equal(out[~broken], want[~broken])
    assert torch.equal(out[5], x[5].to(dev) if with_residual else torch.zeros_like(out[5]))
    grads = torch.autograd.grad(out, leaves, torch.ones_like(out))
    assert torch.isnan(grads[1][broken]).all()
    assert torch.isfinite(grads[1][~broken]).all() and (grads[1][5] == 0).all()
    for i in (0, 2, 3):  # no expert saw the broken tokens
        assert torch.isfinite(grads[i]).all()


@pytest.mark.parametrize("E,k", [(12, 3), (256, 8), (500, 16), (1000, 32)])
@pytest.mark.parametrize("options", [dict(), dict(renormalize=False), dict(score="sigmoid"),
                                     dict(score="sigmoid", renormalize=False), dict(score="given"),
                                     dict(score="given", renormalize=False)])
def test_route_gradient_of_rows_that_are_not_finite(dev, E, k, options):
    z = torch.rand(70, E, generator=gen(E)) + 0.5
    clean = z.to(dev).requires_grad_(True)
    g = torch.randn(70, k, generator=gen(k)).to(dev)
    (want,) = torch.autograd.grad(stk.route(clean, k, **options)[0], [clean], g)
    z[1, E - 1] = math.nan
    z[17, 0] = math.inf
    z[69, E // 2] = math.inf
    z[33] = -math.inf
    leaf = z.to(dev).requires_grad_(True)
    (dz,) = torch.autograd.grad(stk.route(leaf, k, **options)[0], [leaf], g)
    assert torch.isnan(dz[[1, 17, 69]]).all()
    assert (dz[33] == 0).all()
    rest = torch.ones(70, dtype=torch.bool, device=dev)
    rest[[1, 17, 33, 69]] = False
    assert torch.equal(dz[rest], want[rest])


@pytest.mark.parametrize("T,k,N,dtype", [(9, 2, 40, "bf16"), (20, 12, 37, "f16"), (3, 8, 2048, "f32")])
def test_combine_keeps_the_nan_of_dropped_choices_when_asked(dev, T, k, N, dtype):
    y, w, slots, res, dout = base.combine_inputs(T, k, N, dtype, True, 0.3)
    slots[1] = slots[0, k - 1] = -1
    kept = slots >= 0
    slots[kept] = torch.randperm(int(kept.sum()), generator=gen(N)).to(torch.int32)
    w[~kept] = 0.5  # finite: left out as ever
    slots[0, k - 1] = T * k + 3  # no place either
    clean = w.clone()
    w[0, k - 1] = math.nan
    w[1, 0] = math.nan
    args = [t.to(dev) for t in (y, w, slots, res)]
    out = stk.combine(*args, keep_nan=True)
    value, bound = ref.combine(y, clean, slots, res)[0]
    assert torch.isnan(out[:2]).all()
    within(out[2:], value[2:], bound[2:], "out")
    within(stk.combine(*args), value, bound, "out, NaN left out")
    yd = args[0].requires_grad_(True)
    a = torch.autograd.grad(stk.combine(yd, *args[1:], keep_nan=True), [yd], dout.to(dev))[0]
    b = torch.autograd.grad(stk.combine(yd, *args[1:]), [yd], dout.to(dev))[0]
    assert torch.equal(a, b)


def test_layer_with_a_nan_bias_is_nan(dev):
    x, scores, w_up, w_down = (t.to(dev) for t in base.layer_inputs())
    bias = torch.zeros(12, device=dev)
    bias[4] = math.nan
    out, experts = stk.moe(x, scores, w_up, w_down, 3, residual=x, bias=bias)
    assert torch.isnan(out).all() and (experts == -1).all()


# ---- scores and biases at the type's lowest value ---------------------------------

LOWEST = torch.finfo(torch.float32).min


def check_choice(dev, z, k, options):
    want_w, want_e = ref.route(z, k, **options)
    w, e = stk.route(z.to(dev), k, **base.on(options, dev))
    assert torch.equal(e.cpu(), want_e)
    within(w, want_w, want_w.abs() * 1.01 * ref.U32 + 1e-40, "weights")


@pytest.mark.parametrize("E,k", [(8, 6), (60, 8), (256, 8), (512, 16), (1024, 32)])
def test_lowest_score_with_a_lowering_bias_stays_available(dev, E, k):
    # u = z + bias = -4.4e38 is a number (fp32 has none there): chosen after all others, lowest index first
    z = torch.rand(20, E, generator=gen(E))
    z[:, k // 2:] = LOWEST
    bias = torch.zeros(E)
    bias[k // 2:] = -1e38
    check_choice(dev, z, k, dict(score="given", renormalize=False, bias=bias))
    bias[E - 1] = -0.9e38  # now the last is the best of those
    check_choice(dev, z, k, dict(score="given", renormalize=False, bias=bias))


@pytest.mark.parametrize("E,k,groups,open_", [(16, 10, 4, 3), (60, 8, 6, 5), (256, 8, 8, 6), (512, 16, 32, 31),
                                              (1024, 32, 64, 60)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid", "given"])
def test_group_of_lowest_biases_stays_available(dev, E, k, groups, open_, score):
    # a group whose two best are both at the lowest value has a sum (-6.8e38) that orders it last, ties by index
    z = torch.rand(20, E, generator=gen(E)) + 0.5
    size = E // groups
    bias = torch.zeros(E)
    bias[:(groups - 1) * size] = LOWEST
    options = dict(score=score, bias=bias, n_group=groups, topk_group=open_, group_top=2, renormalize=False)
    if size < k:
        check_choice(dev, z, k, options)
    bias[size:2 * size:2] = 0.25  # one or more of a group's two best
    check_choice(dev, z, min(k, 8), options)


@pytest.mark.parametrize("group_top", [1, 2])
def test_groups_of_lowest_scores(dev, group_top):
    z = torch.rand(30, 64, generator=gen(6))
    z[:, 8:40] = LOWEST
    z[3] = LOWEST
    z[4, ::2] = LOWEST
    z[5] = 3e38
    for open_ in (1, 3, 4, 6, 8):
        check_choice(dev, z, 8, dict(score="given", n_group=8, topk_group=open_, group_top=group_top,
                                     renormalize=False))


# ---- many groups --------------------------------------------------------------------

@pytest.mark.parametrize("E,k,groups,open_", [(256, 8, 32, 5), (255, 7, 17, 3), (256, 8, 64, 20), (128, 8, 64, 64),
                                              (512, 16, 32, 9), (512, 12, 64, 11), (510, 16, 17, 4),
                                              (1024, 32, 64, 12), (960, 20, 60, 9), (64, 1, 64, 1)])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_with_many_groups(dev, E, k, groups, open_, group_top, score):
    print("[groups] E=%d k=%d %d of %d top %d %s" % (E, k, open_, groups, group_top, score), flush=True)
    for masked, bias in ((0.0, True), (0.4, False)):
        options = dict(score=score, bias=bias, n_group=groups, topk_group=open_, group_top=group_top, scale=1.5)
        z, options = base.route_inputs(37, E, "f32", options, masked)
        want_w, want_e = ref.route(z, k, **options)
        zd = z.to(dev).requires_grad_(True)
        w, e = stk.route(zd, k, **base.on(options, dev))
        g = torch.randn(37, k, generator=gen(E))
        (dz,) = torch.autograd.grad(w, [zd], g.to(dev))
        assert torch.equal(e.cpu(), want_e)
        within(w, want_w, want_w * 1.01 * ref.U32 + 1e-40, "weights")
        want = ref.route_grad(z, want_e, g, **{n: v for n, v in options.items() if n != "bias"})
        # renormalised: at the chosen only, in fp64; where its parts cancel (k = 1: to 0) some eight fp64 roundings of
        # the parts remain on either side, 8 2^-53 scale |g| each
        parts = 1.5 * g.abs().double().sum(1, keepdim=True) * 2.0 ** -49
        within(dz, want, want.abs() * 1.01 * ref.U32 + parts + ref.tiny(torch.float32), "grad")


# ---- offsets that are not a dispatch's -------------------------------------------

def fenced(shape, dtype, dev, fill):
    """A tensor between two fences of 64 KiB each, and the whole storage."""
    n = math.prod(shape)
    pad = (1 << 16) // torch.empty(0, dtype=dtype).element_size()
    store = torch.full((n + 2 * pad,), fill, dtype=dtype, device=dev)
    return store[pad:pad + n].view(shape), store, pad


@pytest.mark.parametrize("act", ["none", "gelu", "swiglu"])
@pytest.mark.parametrize("E,T,K,N", [(64, 700, 64, 96), (1024, 900, 72, 40), (3, 70, 33, 17), (512, 4096, 264, 264)])
def test_product_with_wrong_offsets_stays_inside(dev, act, E, T, K, N):
    # offsets that fall, leave [0, pairs] or name every row for every second expert: the results mean nothing, and
    # nothing outside them is read (the library checks its own table) or written
    lib = stk._lib.load()
    bf = torch.bfloat16
    code = {"none": 0, "gelu": 2, "swiglu": 3}[act]
    M = 2 * N if act == "swiglu" else N
    x, w = torch.ones(T, K, dtype=bf, device=dev), torch.ones(E, M, K, dtype=bf, device=dev)
    b, dy = torch.ones(E, M, dtype=bf, device=dev), torch.ones(T, N, dtype=bf, device=dev)
    wrong = [[T * (e % 2) for e in range(E + 1)], [T - e for e in range(E + 1)], [-5] * E + [2 ** 31 - 1],
             [(-1) ** e * (2 ** 31 - 1) for e in range(E + 1)], [0] + [T] + [0] * (E - 1), [T] * (E + 1)]
    for case in wrong:
        offsets = torch.tensor(case, dtype=torch.int32, device=dev)
        outs = {n: fenced(s, t, dev, 7.0) for n, (s, t) in dict(
            y=((T, N), bf), z=((T, M), torch.float32), dx=((T, K), bf), dw=((E, M, K), bf), db=((E, M), bf),
            dr=((T, N), bf)).items()}
        p = {n: v[0].data_ptr() for n, v in outs.items()}
        rc = lib.soft_topk_experts_forward(x.data_ptr(), w.data_ptr(), b.data_ptr(), None, 1, offsets.data_ptr(), None,
                                           T, T, E, K, N, code, p["y"], p["z"], None)
        assert rc == 0
        torch.cuda.synchronize()
        need = lib.soft_topk_experts_backward_workspace_bytes(T, E, K, N, code, 0)
        ws, store, pad = fenced((need,), torch.uint8, dev, 7)
        ws_ptr = (ws.data_ptr() + 255) // 256 * 256  # (the fence behind is 255 bytes nearer at most)
        rc = lib.soft_topk_experts_backward(dy.data_ptr(), x.data_ptr(), w.data_ptr(), p["z"], 1, offsets.data_ptr(),
                                            None, None, T, T, 1, E, K, N, code, p["dx"], p["dw"], p["db"], ws_ptr,
                                            need, None)
        assert rc == 0
        torch.cuda.synchronize()
        rc = lib.soft_topk_experts_residual_backward(dy.data_ptr(), 1, offsets.data_ptr(), T, E, N, p["dr"], None)
        assert rc == 0
        torch.cuda.synchronize()
        for n, (t, whole, edge) in outs.items():
            assert (whole[:edge] == 7).all() and (whole[whole.numel() - edge:] == 7).all(), (n, case[:4])
        assert (store[:pad] == 7).all() and (store[store.numel() - pad + 256:] == 7).all()


# ---- more tokens than a launch holds -----------------------------------------------

def test_route_of_more_tokens_than_a_launch_holds(dev):
    # 2^28 rows at 16 lanes a row, 2^26 at 64: 2^32 work-items
    for T, E, k in (((1 << 28) + 5, 1, 1), ((1 << 26) + 9, 18, 17)):
        print("[route] T=%d E=%d k=%d" % (T, E, k), flush=True)
        z = torch.rand(T, E, device=dev, dtype=torch.bfloat16)
        w, e = stk.route_forward(z, k, score="given", renormalize=False)
        at = torch.cat([torch.arange(c - 3, c + 3) for c in (3, 1 << 23, 1 << 24, 1 << 25, 1 << 26)]
                       + [torch.arange(T - 5, T)])
        at = at[at < T]
        want_w, want_e = ref.route(z[at.to(dev)].cpu(), k, score="given", renormalize=False)
        assert torch.equal(e[at.to(dev)].cpu(), want_e) and torch.equal(w[at.to(dev)].cpu().double(), want_w)
        for first in range(0, T, 1 << 24):  # no row is left out
            assert (e[first:first + (1 << 24)] >= 0).all()
        g = w  # a cotangent at hand
        dz = stk.route_backward(g, z, e, score="given", renormalize=False)
        want = ref.route_grad(z[at.to(dev)].cpu(), want_e, g[at.to(dev)].cpu(), score="given", renormalize=False)
        assert torch.equal(dz[at.to(dev)].cpu().double(), want)
        if E == 1:
            assert torch.equal(dz, z)
        del z, w, e, g, dz
        torch.cuda.empty_cache()


def test_combine_of_more_tokens_than_a_launch_holds(dev):
    # 256 lanes a token: 2^24 tokens are 2^32 work-items
    T, N, P = (1 << 24) + 7, 1032, 500
    slots = torch.full((T, 1), -1, dtype=torch.int32)
    at = torch.cat([torch.arange(c, c + 60) for c in (0, (1 << 23) - 30, (1 << 24) - 55)])
    at = torch.cat([at, torch.arange(T - 2, T)])
    slots[at, 0] = torch.randperm(len(at), generator=gen(60)).to(torch.int32)
    y = torch.randn(P, N, generator=gen(61)).to(torch.bfloat16)
    w = torch.rand(T, 1, generator=gen(62))
    yd, wd, sd = y.to(dev), w.to(dev), slots.to(dev)
    out = stk.combine_forward(yd, wd, sd)
    value, bound = ref.combine(y, w[at], slots[at], None)[0]
    within(out[at.to(dev)], value, bound, "out")
    assert (out[100:1000] == 0).all() and (out[(1 << 23) + 100:(1 << 23) + 1000] == 0).all()
    dout = out.fill_(0)
    some = torch.randn(len(at), N, generator=gen(63)).to(torch.bfloat16)
    dout[at.to(dev)] = some.to(dev)
    dy, dw = stk.combine_backward(dout, yd, wd, sd)
    _, want_dy, want_dw = ref.combine(y, w[at], slots[at], None, some)
    within(dy, *want_dy, "dy")
    assert (dy[len(at):] == 0).all()
    within(dw[at.to(dev)], *want_dw, "dw")
    assert (dw[100:1000] == 0).all()
    del out, dout
    torch.cuda.empty_cache()


def test_product_of_more_rows_than_31_bits_of_elements(dev):
    R, K, N = (1 << 29) + 77, 8, 8  # 8.6e9 bytes of x, 4.3e9 elements
    x = torch.zeros(R, K, dtype=torch.bfloat16, device=dev)
    at = torch.cat([torch.arange(c, c + 9) for c in (0, 1 << 28, (1 << 29) - 4, R - 9)])
    small = torch.randn(len(at), K, generator=gen(64)).to(torch.bfloat16)
    x[at.to(dev)] = small.to(dev)
    w = torch.randn(1, N, K, generator=gen(65)).to(torch.bfloat16)
    off = torch.tensor([0, R], dtype=torch.int32)
    y = stk.experts_product(x, w.to(dev), stk.Dispatch(off.to(dev)), act="silu")
    few = torch.tensor([0, len(at)], dtype=torch.int32)
    within(y[at.to(dev)], *ref.product(small, w, few, None, None, "silu", None)[0], "y")
    assert (y[1000:100000] == 0).all()
    del y
    dy = torch.zeros(R, N, dtype=torch.bfloat16, device=dev)
    dsmall = torch.randn(len(at), N, generator=gen(66)).to(torch.bfloat16)
    dy[at.to(dev)] = dsmall.to(dev)
    dx, dw, db = stk.experts_backward(dy, x, w.to(dev), stk.Dispatch(off.to(dev)), want=(True, True, True))
    _, want_dx, want_dw, want_db = ref.product(small, w, few, None, None, "none", None, dsmall)
    within(dx[at.to(dev)], *want_dx, "dx")
    within(dw, *want_dw, "dw")
    within(db, *want_db, "db")
    del x, dy, dx
    torch.cuda.empty_cache()


# ---- what the forward keeps --------------------------------------------------------

def test_product_keeps_no_z_for_a_residual_alone(dev):
    x, w, offsets, rows, slots, b, res, dy = base.product_inputs(4000, 2, 4, 64, 512, "silu", "bf16", True, True, True,
                                                                 0.1)
    plan = stk.Dispatch(offsets.to(dev), rows.to(dev), slots.to(dev))
    x, w, b, res = (t.to(dev) for t in (x, w, b, res))
    leaf = res.requires_grad_(True)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    y = stk.experts_product(x, w, plan, bias=b, act="silu", residual=leaf)
    held = torch.cuda.memory_allocated() - before
    assert held < y.numel() * y.element_size() + (1 << 20)  # y alone: z would be twice its size
    (grad,) = torch.autograd.grad(y, [leaf], dy.to(dev))
    assert torch.equal(grad.cpu(), residual_gradient(dy, offsets))
    # any other leaf keeps it
    for i, t in enumerate((x, w, b)):
        t.requires_grad_(True)
        y = stk.experts_product(x, w, plan, bias=b, act="silu", residual=leaf)
        (grad,) = torch.autograd.grad(y, [t], dy.to(dev))
        t.requires_grad_(False)
        want = ref.product(x.cpu(), w.cpu(), offsets, rows, b.cpu(), "silu", res.detach().cpu(), dy)[1 + i]
        within(grad, *want, "leaf %d" % i)


def test_combine_of_a_row_of_nearly_31_bits(dev):
    # the step behind the last of 2^31 - 8 columns passes 2^31
    N = (1 << 31) - 8
    y = torch.zeros(2, N, dtype=torch.bfloat16, device=dev)
    at = torch.cat([torch.arange(40), torch.arange((1 << 30) - 20, (1 << 30) + 20), torch.arange(N - 40, N)]).to(dev)
    small = torch.randn(2, len(at), generator=gen(67)).to(torch.bfloat16)
    y[:, at] = small.to(dev)
    w = torch.tensor([[0.75, 0.5]])
    slots = torch.tensor([[1, 0]], dtype=torch.int32)
    out = stk.combine_forward(y, w.to(dev), slots.to(dev))
    within(out[:, at], *ref.combine(small, w, slots, None)[0], "out")
    assert (out[0, 1000:1 << 20] == 0).all()
    dy, dw = stk.combine_backward(out, y, w.to(dev), slots.to(dev))
    dout = out[:, at].cpu()
    _, want_dy, want_dw = ref.combine(small, w, slots, None, dout)
    within(dy[:, at], *want_dy, "dy")
    within(dw, *want_dw, "dw")
    del y, out, dy
    torch.cuda.empty_cache()
