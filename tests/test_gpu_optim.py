"""The training step's update on the GPU against oracle/optim.py.

Tolerances (u = 2^-24): m, v, sqrt(v), and with them every 8-bit state: bit for bit, since each rounding is part of the
definition.  A new fp32 parameter: two constants and up to three roundings in param (1 - lr decay), and five constants and
up to eight roundings in the rest (sqrt(v), its product, the sum with eps, the quotient, its product), so
4 u |param| + 12 u |update| and the last rounding, u |new|.  A bf16 one: between what the random bits make of the two ends of
that range, nearly always one value.  The bf16 copy: the new parameter's
nearest, bit for bit.  The norm: fp64, one rounding."""
import numpy as np
import pytest
import torch

import fp8_compression_tensor_taco_amd as taco
from oracle import linear as ol
from oracle import optim as oo
from test_gpu_linear import U, f64, guarded, survived

pytestmark = pytest.mark.gpu
HYPER = dict(lr=3e-3, step=7, betas=(0.9, 0.99), eps=1e-8)
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


def make(sizes, params, grads, bits, seed=0):
    """CPU tensors of a list: parameters, gradients, states as a training has them, a few elements never touched."""
    rng = np.random.default_rng(seed)
    out = dict(params=[], grads=[], m=[], v=[])
    for i, n in enumerate(sizes):
        width = 1e-3 * np.exp(rng.standard_normal())
        p, g = 0.02 * rng.standard_normal(n), width * rng.standard_normal(n)
        m, r = 0.3 * width * rng.standard_normal(n), width * np.exp(rng.standard_normal(n))
        for x in (g, m, r):
            x[3::17] = 0
        out["params"].append(torch.from_numpy(p).to(DTYPES[params]))
        out["grads"].append(torch.from_numpy(g).to(DTYPES[grads]))
        if bits == 32:
            out["m"].append(torch.from_numpy(m.astype(np.float32)))
            out["v"].append(torch.from_numpy((r * r).astype(np.float32)))
        else:
            for x, to in ((m, out["m"]), (r, out["v"])):
                q, s = ol.quantize_rows(x[None])
                to.append((torch.from_numpy(q[0]), torch.from_numpy(s[0])))
    return out


def to_gpu(x):
    return [to_gpu(v) for v in x] if isinstance(x, list) else tuple(v.cuda() for v in x) if isinstance(x, tuple) else x.cuda()


def numpy_state(s):
    return tuple(v.cpu().numpy() for v in s) if isinstance(s, tuple) else s.cpu().numpy()


def check_parameter(got, new, p, lr, decay, half=None):
    """fp64 new parameters before their rounding against the GPU's."""
    moved = np.abs(new - p * (1 - lr * decay))
    err = 4 * U * np.abs(p) + 12 * U * moved + U * np.abs(new)
    if got.dtype == torch.float32:
        assert (np.abs(f64(got) - new) <= err).all()
        return
    # for given random bits the rounding is monotonic, so the result lies between those of the ends
    lo, hi = (np.copysign(oo.stochastic(np.abs(x), 7, -126, half), x) for x in (new - err, new + err))
    d = f64(got)
    assert ((d >= lo) & (d <= hi)).all()
    assert np.sum(lo != hi) <= 3 + 0.01 * d.size          # nearly every element is decided


def check_step(given, gpu, copies, hyper, decay, factor=1.0, seed=0):
    for i, p in enumerate(given["params"]):
        n = p.numel()
        if n == 0:
            continue
        m, v = (numpy_state(given[k][i]) for k in ("m", "v"))
        new, want_m, want_v = oo.adamw(f64(p), given["grads"][i].float().numpy(), m, v, decay=decay, factor=factor, index=i,
                                       seed=seed, **hyper)
        for got, want in ((gpu["m"][i], want_m), (gpu["v"][i], want_v)):
            if isinstance(want, tuple):
                assert all((a.cpu().numpy() == b).all() for a, b in zip(got, want)), i
            else:
                assert (got.cpu().numpy() == want).all(), i
        check_parameter(gpu["params"][i], new, f64(p), hyper["lr"], decay, oo.random_halves(n, i, hyper["step"], seed)[2])
        if copies and copies[i] is not None:
            assert torch.equal(copies[i], gpu["params"][i].to(torch.bfloat16))


SIZES = [[1], [5], [127, 128, 129], [1000], [2048, 2047, 2049, 4100], [3, 0, 20000, 1], [17] * 49, [70001]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("params,grads", [("fp32", "fp32"), ("fp32", "bf16"), ("bf16", "fp32"), ("bf16", "bf16")])
def test_step(params, grads, bits, sizes):
    sizes = [n for n in sizes if n or bits == 32]
    given = make(sizes, params, grads, bits, len(sizes))
    gpu = {k: to_gpu(v) for k, v in given.items()}
    copies = [torch.full((n,), 7.0, dtype=torch.bfloat16).cuda() for n in sizes] if params == "fp32" else None
    before = [g.clone() for g in gpu["grads"]]
    assert taco.adamw_step(gpu["params"], gpu["grads"], gpu["m"], gpu["v"], weight_decay=0.1, copies=copies, seed=99, **HYPER) is None
    check_step(given, gpu, copies, HYPER, 0.1, seed=99)
    assert all(torch.equal(a, b) for a, b in zip(before, gpu["grads"]))


def test_mixed_list():
    """Types, states and copies of all kinds in one call, over several launches."""
    kinds = [(p, g, b) for p in ("fp32", "bf16") for g in ("fp32", "bf16") for b in (8, 32)] * 14
    parts = [make([37 + 11 * i], *kind, seed=i) for i, kind in enumerate(kinds)]
    given = {k: [p[k][0] for p in parts] for k in parts[0]}
    gpu = {k: to_gpu(v) for k, v in given.items()}
    copies = [torch.zeros(p.numel(), dtype=torch.bfloat16).cuda() if i % 3 and p.dtype == torch.float32 else None
              for i, p in enumerate(gpu["params"])]
    taco.adamw_step(gpu["params"], tuple(gpu["grads"]), gpu["m"], gpu["v"], weight_decay=0.0, copies=copies, seed=2 ** 63 + 5, **HYPER)
    check_step(given, gpu, copies, HYPER, 0.0, seed=2 ** 63 + 5)


@pytest.mark.parametrize("bits", [8, 32])
def test_training(bits):
    """Many steps from nothing, against the oracle's own course."""
    rng = np.random.default_rng(0)
    n = 3000
    p0 = torch.from_numpy(rng.standard_normal(n)).float()
    p, copy = p0.cuda(), torch.zeros(n, dtype=torch.bfloat16).cuda()
    m, v = taco.adamw_state(p, bits)
    want_m, want_v, want = numpy_state(m), numpy_state(v), f64(p0)
    for step in range(1, 21):
        g = torch.from_numpy(rng.standard_normal(n) * 10.0 ** rng.integers(-6, 3)).float()
        taco.adamw_step([p], [g.cuda()], [m], [v], lr=1e-2, step=step, betas=(0.9, 0.95), weight_decay=0.1, copies=[copy], seed=step)
        want, want_m, want_v = oo.adamw(want, g.numpy(), want_m, want_v, lr=1e-2, step=step, betas=(0.9, 0.95), eps=1e-8, decay=0.1,
                                        seed=step)
    for got, w in ((m, want_m), (v, want_v)):
        assert all((a == b).all() for a, b in zip(numpy_state(got), w)) if bits == 8 else (numpy_state(got) == w).all()
    # each step adds at most 4 u |p| + 12 u |update| + u |p|; |p| stays below 6 and an update below 4 lr
    assert np.abs(f64(p) - want).max() <= 20 * (5 * 6 + 12 * 0.04) * U
    assert torch.equal(copy, p.to(torch.bfloat16))


def test_rate_step_and_factor_on_the_device():
    given = make([300, 5000], "fp32", "fp32", 8)
    lr, step, factor = torch.tensor([2e-3]), torch.tensor([1234567]), torch.tensor([0.37])
    gpu = {k: to_gpu(v) for k, v in given.items()}
    taco.adamw_step(gpu["params"], gpu["grads"], gpu["m"], gpu["v"], lr=lr.cuda(), step=step.cuda(), grad_scale=factor.cuda(),
                    betas=(0.9, 0.999), weight_decay=0.1, seed=4)
    hyper = dict(lr=float(lr), step=1234567, betas=(0.9, 0.999), eps=1e-8)
    check_step(given, gpu, None, hyper, 0.1, factor=factor.item(), seed=4)
    # numbers in their places give the same, bit for bit
    for kw in (dict(lr=float(lr), step=1234567), dict(lr=lr.cuda(), step=1234567), dict(lr=float(lr), step=step.cuda()[0])):
        other = {k: to_gpu(v) for k, v in given.items()}
        taco.adamw_step(other["params"], other["grads"], other["m"], other["v"], grad_scale=factor.cuda()[0], betas=(0.9, 0.999),
                        weight_decay=0.1, seed=4, **kw)
        assert all(torch.equal(a, b) for a, b in zip(other["params"], gpu["params"]))
        assert all(torch.equal(x, y) for a, b in zip(other["m"] + other["v"], gpu["m"] + gpu["v"]) for x, y in zip(a, b))


@pytest.mark.parametrize("now,same_as", [(0, 1), (-3, 1), (1, 1)])
def test_a_step_on_the_device_is_one_at_least(now, same_as):
    given = make([700], "fp32", "fp32", 8)
    got = []
    for step in (torch.tensor([now]).cuda(), same_as):
        gpu = {k: to_gpu(v) for k, v in given.items()}
        taco.adamw_step(gpu["params"], gpu["grads"], gpu["m"], gpu["v"], lr=1e-3, step=step)
        got.append(gpu)
    assert torch.equal(got[0]["params"][0], got[1]["params"][0]) and torch.equal(got[0]["m"][0][0], got[1]["m"][0][0])


@pytest.mark.parametrize("factor", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("bits", [8, 32])
def test_a_factor_that_is_not_finite_leaves_the_step_out(bits, factor):
    given = make([300, 5000], "fp32", "bf16", bits)
    gpu = {k: to_gpu(v) for k, v in given.items()}
    copies = [torch.full((p.numel(),), 3.0, dtype=torch.bfloat16).cuda() for p in gpu["params"]]
    taco.adamw_step(gpu["params"], gpu["grads"], gpu["m"], gpu["v"], copies=copies, grad_scale=torch.tensor([factor]).cuda(), **HYPER)
    for k in given:
        for a, b in zip(given[k], gpu[k]):
            assert all(torch.equal(x, y.cpu()) for x, y in zip(a, b)) if isinstance(a, tuple) else torch.equal(a, b.cpu())
    assert all((c == 3).all() for c in copies)


@pytest.mark.parametrize("params", ["fp32", "bf16"])
def test_non_finite_gradients(params):
    """fp32 states: the element alone; 8-bit states: its block is NaN from the next step on."""
    given = {bits: make([1000], params, "fp32", bits) for bits in (8, 32)}
    for bits, one in given.items():
        one["grads"][0][200], one["grads"][0][700] = float("nan"), float("inf")
        gpu = {k: to_gpu(v) for k, v in one.items()}
        taco.adamw_step(gpu["params"], gpu["grads"], gpu["m"], gpu["v"], **HYPER)
        # m and v are infinite at 700: their quotient is NaN
        nan = torch.isnan(gpu["params"][0]).cpu()
        assert nan[200] and nan[700] and int(nan.sum()) == 2
        if bits == 8:
            for q, s in (gpu["m"][0], gpu["v"][0]):
                assert (s.cpu() == 255).nonzero().flatten().tolist() == [1, 5]
                assert (q[128:256] == 0x7F).all() and (q[640:768] == 0x7F).all() and not (q[:128] == 0x7F).any()
            taco.adamw_step(gpu["params"], [torch.zeros(1000).cuda()], gpu["m"], gpu["v"], **HYPER)
            nan = torch.isnan(gpu["params"][0]).cpu()
            assert nan[128:256].all() and nan[640:768].all() and int(nan.sum()) == 256
        else:
            assert torch.isnan(gpu["m"][0]).nonzero().flatten().tolist() == [200] and torch.isinf(gpu["m"][0][700])


def test_extreme_values():
    """Moments at the ends of fp32's range, blocks of one value, and states whose scale is the least."""
    n = 128 * 6
    g = np.zeros(n, np.float32)
    g[:128], g[128:256], g[256:384] = 1e18, 1e-22, 1e-38
    g[384:512] = np.logspace(-40, 15, 128)
    g[512] = 5.0
    g[640:] = -np.logspace(-10, 10, 128)
    m, r = np.zeros(n), np.abs(g.astype(float)) * 0.5
    given = dict(params=[torch.ones(n)], grads=[torch.from_numpy(g)], m=[], v=[])
    for x, to in ((m, given["m"]), (r, given["v"])):
        q, s = ol.quantize_rows(x[None])
        to.append((torch.from_numpy(q[0]), torch.from_numpy(s[0])))
    gpu = {k: to_gpu(v) for k, v in given.items()}
    taco.adamw_step(gpu["params"], gpu["grads"], gpu["m"], gpu["v"], weight_decay=0.0, seed=3, **HYPER)
    check_step(given, gpu, None, HYPER, 0.0, seed=3)


def test_lying_anywhere():
    """Parameters, gradients, fp32 states and copies at any element's place; nothing beside them is written."""
    for params, bits in (("fp32", 32), ("fp32", 8), ("bf16", 8)):
        for off in (1, 2, 3):
            given = make([1003, 130], params, "bf16", bits, off)
            want = {k: to_gpu(v) for k, v in given.items()}
            want_copies = [torch.zeros(n, dtype=torch.bfloat16).cuda() for n in (1003, 130)] if params == "fp32" else None
            taco.adamw_step(want["params"], want["grads"], want["m"], want["v"], copies=want_copies, **HYPER)
            held = []

            def moved(t):
                if isinstance(t, tuple):
                    return tuple(place(x, 0) for x in t)
                return place(t, off)

            def place(t, by):
                whole, view = guarded((t.numel() + by,), t.dtype)
                view[by:].copy_(t)
                held.append((whole, view[:by].clone(), view, by))
                return view[by:]

            gpu = {k: [moved(t) for t in to_gpu(v)] for k, v in given.items()}
            copies = [place(torch.zeros_like(c), off) for c in want_copies] if want_copies else None
            taco.adamw_step(gpu["params"], gpu["grads"], gpu["m"], gpu["v"], copies=copies, **HYPER)
            for k in ("params", "m", "v"):
                for a, b in zip(gpu[k], want[k]):
                    assert all(torch.equal(x, y) for x, y in zip(a, b)) if isinstance(a, tuple) else torch.equal(a, b)
            assert not copies or all(torch.equal(a, b) for a, b in zip(copies, want_copies))
            assert all(survived(w) and torch.equal(view[:by].view(torch.uint8), kept.view(torch.uint8)) for w, kept, view, by in held)


def test_strided_gradients_and_shapes():
    p = torch.randn(40, 60, device="cuda")
    g = torch.randn(60, 40, device="cuda").t()
    a, b = p.clone(), p.clone()
    sa, sb = taco.adamw_state(p, 8), taco.adamw_state(p, 8)
    taco.adamw_step([a], [g], [sa[0]], [sa[1]], **HYPER)
    taco.adamw_step([b], [g.contiguous()], [sb[0]], [sb[1]], **HYPER)
    assert torch.equal(a, b) and torch.equal(sa[1][0], sb[1][0])


def test_refusals():
    p = torch.randn(4, 300, device="cuda")
    m, v = taco.adamw_state(p)
    (mq, vq), h = taco.adamw_state(p, 8), p.to(torch.bfloat16)
    good = dict(params=[p], grads=[p.clone()], m=[m], v=[v])
    bad = [dict(params=[p.half()]), dict(params=[p[:, ::2]]), dict(grads=[p.double()]), dict(grads=[p[:3]]), dict(grads=[p.flatten()]),
           dict(grads=[]), dict(m=[m.to(torch.bfloat16)]), dict(m=[m[:3]]), dict(m=[mq]), dict(m=[mq[0]]), dict(m=[list(mq)], v=[vq]),
           dict(m=[(mq[0][:-1], mq[1])], v=[vq]), dict(m=[(mq[0], mq[1][:-1])], v=[vq]), dict(copies=[p.clone()]), dict(copies=[]),
           dict(copies=h), dict(params=[h], copies=[h.clone()]), dict(lr="fast"), dict(step=1.5), dict(lr=torch.zeros(2).cuda()),
           dict(step=torch.ones(1).cuda()), dict(lr=torch.ones(1)), dict(grad_scale=0.5), dict(grad_scale=torch.ones(2).cuda()),
           dict(grad_scale=torch.ones(1, dtype=torch.float64).cuda()), dict(grads=[p.cpu()]), dict(params=[None])]
    for over in bad:
        with pytest.raises(ValueError):
            taco.adamw_step(**{**good, "lr": 1e-3, "step": 1, **over})
    for over, name in ((dict(grads=[p]), "ALIAS"), (dict(m=[v]), "ALIAS"), (dict(m=[p]), "ALIAS"), (dict(step=0), "SHAPE"),
                       (dict(betas=(1.0, 0.9)), "SHAPE"), (dict(eps=-1.0), "SHAPE"), (dict(lr=float("nan")), "SHAPE"),
                       (dict(params=[p, p], grads=[p.clone()] * 2, m=[m, m.clone()], v=[v, v.clone()]), "ALIAS")):
        with pytest.raises(taco.TacoError) as e:
            taco.adamw_step(**{**good, "lr": 1e-3, "step": 1, **over})
        assert e.value.name == "TACO_ERR_" + name
    # gradients may share memory
    g = p.clone()
    q = p.clone()
    taco.adamw_step([p, q], [g, g], [m, m.clone()], [v, v.clone()], lr=1e-3, step=1)
    assert torch.equal(p, q)


# ------------------------------------------------------------------------------------ norm

@pytest.mark.parametrize("sizes", SIZES + [[100] * 200, [5000000, 3], [64 * 4096 * 5 + 7]], ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "both"])
def test_norm(dtype, sizes):
    rng = np.random.default_rng(len(sizes))
    grads = [torch.from_numpy(rng.standard_normal(n) * 1e-3).to(DTYPES["bf16" if dtype == "bf16" or (dtype == "both" and i % 2) else "fp32"])
             for i, n in enumerate(sizes)]
    want = np.sqrt(sum((f64(g) ** 2).sum() for g in grads))
    given = [g.cuda() for g in grads]
    for max_norm in (None, 1e-4, 1e9, want * (1 + 1e-3)):
        out = taco.gradient_norm(given, max_norm)
        assert out.shape == (2,) and out.dtype == torch.float32
        factor = 1.0 if max_norm is None or want <= max_norm else max_norm / want
        assert abs(float(out[0]) - want) <= 1.001 * U * want and abs(float(out[1]) - factor) <= 1.001 * U * factor
        assert torch.equal(out, taco.gradient_norm(given, max_norm))


def test_norm_range_and_non_finite():
    for value, n in ((3e38, 1), (1e30, 1000), (1e-30, 1000), (1e-45, 5), (0.0, 100)):
        x = torch.full((n,), value).cuda()
        want = float(x[0].double()) * n ** 0.5
        got = f64(taco.gradient_norm([x], 1.0))
        assert abs(got[0] - want) <= 1.001 * U * want + 2.0 ** -150 and abs(got[1] - min(1, 1 / want if want else 1)) <= U
    for bad in (float("nan"), float("inf"), -float("inf")):
        x = torch.zeros(5000).cuda()
        x[4999] = bad
        out = taco.gradient_norm([torch.ones(10).cuda(), x], 1.0)
        assert not torch.isfinite(out[0]) and torch.isnan(out[1])
    out = taco.gradient_norm([torch.full((100,), 3e38).cuda()], 1.0)         # beyond fp32
    assert torch.isinf(out[0]) and torch.isnan(out[1])
    assert taco.gradient_norm([torch.zeros(0).cuda()], 1.0).tolist() == [0.0, 1.0]


def test_norm_layouts_workspace_and_refusals():
    x = torch.randn(300, 70, device="cuda")
    flat = torch.randn(1001, device="cuda")
    for view in (x.t(), x[:, ::2], flat[1:], flat.to(torch.bfloat16)[3:]):
        assert torch.equal(taco.gradient_norm([view, x]), taco.gradient_norm([view.contiguous().clone(), x]))
    need = taco.gradient_norm_workspace_bytes(2)
    whole, ws = guarded((need,), torch.uint8)
    ws.fill_(0xFF)
    held, out = guarded((2,), torch.float32)
    got = taco.gradient_norm([x, flat], 0.5, out=out, workspace=ws)
    assert got.data_ptr() == out.data_ptr() and torch.equal(got, taco.gradient_norm([x, flat], 0.5)) and survived(whole) and survived(held)
    for bad in (lambda: taco.gradient_norm([x.half()]), lambda: taco.gradient_norm([x, x.cpu()]), lambda: taco.gradient_norm([x, 3]),
                lambda: taco.gradient_norm([x], out=torch.zeros(3).cuda())):
        with pytest.raises(ValueError):
            bad()
    for bad, name in ((lambda: taco.gradient_norm([x], 0.0), "SHAPE"), (lambda: taco.gradient_norm([x], workspace=ws[:need - 8]), "WORKSPACE"),
                      (lambda: taco.gradient_norm([flat], out=flat[:2]), "ALIAS")):
        with pytest.raises(taco.TacoError) as e:
            bad()
        assert e.value.name == "TACO_ERR_" + name


# ------------------------------------------------------------------------- streams, graphs, runs

def test_another_stream():
    given = make([3000, 70], "fp32", "fp32", 8)
    stream = torch.cuda.Stream()
    runs = []
    for s in (None, stream):
        gpu = {k: to_gpu(v) for k, v in given.items()}
        torch.cuda.synchronize()
        norm = taco.gradient_norm(gpu["grads"], 0.01, stream=s)
        taco.adamw_step(gpu["params"], gpu["grads"], gpu["m"], gpu["v"], grad_scale=norm[1:], stream=s, **HYPER)
        torch.cuda.synchronize()
        runs.append([norm, *gpu["params"], *(x for k in ("m", "v") for t in gpu[k] for x in t)])
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_graph_of_a_clipped_step():
    """Norm and step captured once, replayed with new gradients, rates and steps; eager steps of the same between."""
    sizes = [40, 5000, 129] * 20
    given = make(sizes, "fp32", "fp32", 8)
    graph_side, eager = ({k: to_gpu(v) for k, v in given.items()} for _ in range(2))
    copies = [[torch.zeros(n, dtype=torch.bfloat16).cuda() for n in sizes] for _ in range(2)]
    lr, step = torch.tensor([1e-3]).cuda(), torch.tensor([1]).cuda()

    def run(s, c):
        norm = taco.gradient_norm(s["grads"], 0.05)
        taco.adamw_step(s["params"], s["grads"], s["m"], s["v"], lr=lr, step=step, grad_scale=norm[1:], copies=c, seed=8)
        return norm

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run({k: to_gpu(v) for k, v in given.items()}, [c.clone() for c in copies[0]])
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = run(graph_side, copies[0])
    for replay in range(4):
        lr.fill_(1e-3 * (replay + 1))
        step.fill_(replay + 1)
        for a, b in zip(graph_side["grads"], eager["grads"]):
            b.normal_().mul_(0.01 if replay != 2 else float("inf"))          # the third step is left out
            a.copy_(b)
        want = run(eager, copies[1])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, want) or replay == 2 and torch.isnan(held[1]) and torch.isnan(want[1])
        for a, b in zip(graph_side["params"] + copies[0], eager["params"] + copies[1]):
            assert torch.equal(a, b) and torch.isfinite(a).all(), replay
        for a, b in zip(graph_side["m"] + graph_side["v"], eager["m"] + eager["v"]):
            assert all(torch.equal(x, y) for x, y in zip(a, b)), replay
