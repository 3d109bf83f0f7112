"""The MXFP4 mixture-of-experts layer on the GPU against the FP64 oracle.

Tolerance, element by element. With A = sum_e p_e |h_e| |W2_e| (magnitudes
throughout), the error of y is at most
  * A * (2^-11 + relative error of h): h enters the last product rounded to
    fp16's 11 bits;
  * h's own error: gate and up are FP32 sums of exact products with at most
    (H / 32 + 24) 2^-23 (|x| |W|) error each, carried through silu(g) u
    (|silu'| <= 1.1, |silu(g)| <= |g|);
  * FP32 sums over I and k and the softmax: (I / 32 + 32) 2^-23 A;
  * the bf16 result: half a unit in the last of 8 bits, at most 2^-8 |y|,
    and half of bf16's smallest number, 2^-134, where y is below its range.
The routing is compared exactly: the inputs keep every token's k-th and
(k+1)-th logit at least 1e-4 apart, far above the logits' FP32 error.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import weight_only_int4_gb300 as w4  # noqa: E402
from gpu_util import torch_to_f64  # noqa: E402
from oracle import mxfp4_ops_oracle as Q  # noqa: E402

pytestmark = pytest.mark.gpu


class Case:
    """Random experts (uniform codes, weights of a few hundredths) and a router whose choices are clear."""

    def __init__(self, T, E, k, H, I, renorm=True, seed=0, xscale=1.0, skew=0.0, lo=118, hi=121):
        rng = np.random.default_rng([seed, T, E, k, H, I])
        self.k, self.renorm, self.T, self.E, self.H, self.I = k, renorm, T, E, H, I
        self.c13 = rng.integers(0, 16, size=(E, H, 2 * I)).astype(np.uint8)
        self.c2 = rng.integers(0, 16, size=(E, I, H)).astype(np.uint8)
        self.e13 = rng.integers(lo, hi + 1, size=(E, H // 32, 2 * I)).astype(np.uint8)
        self.e2 = rng.integers(lo, hi + 1, size=(E, I // 32, H)).astype(np.uint8)
        router = rng.standard_normal((E, H)) / np.sqrt(H) / xscale
        x = rng.standard_normal((T, H)) * xscale
        if skew:                    # most tokens prefer the same experts
            x += skew * np.sqrt(H) * xscale * xscale * router[: max(1, k)].sum(axis=0)
        self.router = torch.from_numpy(router).to(torch.bfloat16)
        self.x = torch.from_numpy(x).to(torch.bfloat16)
        self.settle()

    def settle(self):
        """Redraws tokens whose choice is not clear by 1e-4."""
        rng = np.random.default_rng(7)
        for _ in range(50):
            l = np.sort(self.logits(), axis=1)[:, ::-1]
            gap = l[:, self.k - 1] - l[:, self.k] if self.k < self.E else np.full(self.T, 1.0)
            close = np.nonzero(gap < 1e-4)[0]
            if not len(close):
                return
            for t in close:
                self.x[t] = torch.from_numpy(rng.standard_normal(self.H) * float(self.x[t].double().std())
                                             ).to(torch.bfloat16)
        raise AssertionError("no clear routing found")

    def logits(self):
        return self.x.double().numpy() @ self.router.double().numpy().T

    def device(self):
        pack = lambda c: torch.from_numpy(np.ascontiguousarray(
            np.stack([Q.words(m, 0) for m in c])).view(np.int32)).cuda()
        return (self.x.cuda(), self.router.cuda(), pack(self.c13), torch.from_numpy(self.e13).cuda(), pack(self.c2),
                torch.from_numpy(self.e2).cuda())

    def reference(self):
        """(y, bound) in FP64."""
        x, router = self.x.double().numpy(), self.router.double().numpy()
        idx, p = Q.route(x @ router.T, self.k, self.renorm)
        y, bound = np.zeros_like(x), np.zeros_like(x)
        for e in range(self.E):
            t, s = np.nonzero(idx == e)
            if not len(t):
                continue
            w13, w2 = Q.values(self.c13[e], self.e13[e], 0), Q.values(self.c2[e], self.e2[e], 0)
            gu, mag = x[t] @ w13, np.abs(x[t]) @ np.abs(w13)
            g, u = gu[:, :self.I], gu[:, self.I:]
            with np.errstate(over="ignore"):
                silu = g / (1 + np.exp(-g))
            h = silu * u
            d = (self.H / 32 + 24) * 2.0 ** -23 * mag
            dh = 1.1 * d[:, :self.I] * np.abs(u) + np.abs(silu) * d[:, self.I:] + np.abs(h) * 2.0 ** -20
            q = p[t, s][:, None]
            y[t] += q * (h @ w2)
            a = np.abs(h) @ np.abs(w2)
            bound[t] += q * (a * (2.0 ** -11 + (self.I / 32 + 32) * 2.0 ** -23) + dh @ np.abs(w2))
        return y, bound + 2.0 ** -8 * (np.abs(y) + bound) + 2.0 ** -134


def run(case, **kw):
    return w4.mxfp4_moe(*case.device(), case.k, renormalize=case.renorm, **kw)


def check(case, what=""):
    T, H = case.T, case.H
    buf = torch.full((T * H + 512,), -1536.0, dtype=torch.bfloat16, device="cuda")
    y = buf[256:-256].view(T, H)
    dev = case.device()
    w4.mxfp4_moe(*dev, case.k, renormalize=case.renorm, out=y)
    again = w4.mxfp4_moe(*dev, case.k, renormalize=case.renorm)
    assert w4.device_status() == w4.OK
    assert torch.all(buf[:256] == -1536.0) and torch.all(buf[-256:] == -1536.0), "write outside the output"
    assert torch.equal(y, again), "two calls differ"
    ref, bound = case.reference()
    got = torch_to_f64(y)
    assert np.all(np.isfinite(got)), what
    err = np.abs(got - ref)
    assert np.all(err <= bound), f"{what}: worst ratio {(err / bound).max():.2f}, max err {err.max():.3e}"


@pytest.mark.parametrize("T,E,k,H,I", [
    (1, 1, 1, 32, 32),          # the smallest layer
    (1, 8, 2, 64, 96),
    (2, 3, 3, 96, 32),          # every expert chosen
    (7, 9, 3, 544, 352),        # odd everything; H % 64 == 32: half a last column block
    (1, 32, 4, 2048, 1024),
    (5, 256, 16, 320, 64),      # the most experts and choices
    (16, 64, 8, 512, 256),
    (33, 17, 5, 288, 160),
    (64, 12, 2, 256, 288),
    (64, 40, 8, 1056, 224),
])
@pytest.mark.parametrize("renorm", [True, False])
def test_layer(T, E, k, H, I, renorm):
    check(Case(T, E, k, H, I, renorm), (T, E, k, H, I))


@pytest.mark.parametrize("T,E,k", [(16, 4, 1), (17, 4, 1), (48, 6, 2), (64, 1, 1), (64, 2, 2), (64, 16, 4)])
def test_crowded_experts(T, E, k):
    """More tokens on one expert than a group holds, down to all of them on every expert."""
    check(Case(T, E, k, 320, 128, seed=3, skew=1.0), (T, E, k))


@pytest.mark.parametrize("xscale", [2.0 ** -100, 2.0 ** -12, 2.0 ** 9, 2.0 ** 24])
def test_activation_range(xscale):
    """x far outside the fp16 range; with large x, h spans many powers of two."""
    check(Case(6, 8, 2, 288, 160, seed=4, xscale=xscale), xscale)


def test_runs_of_very_different_magnitude():
    """Gate and up columns whose weights differ by 2^40 between the 32-column runs of h."""
    case = Case(5, 4, 2, 160, 256, seed=5)
    rng = np.random.default_rng(5)
    run_shift = rng.integers(-20, 21, size=case.I // 32).repeat(32)
    case.e13[:, :, case.I:] = np.clip(case.e13[:, :, case.I:].astype(int) + run_shift, 60, 200).astype(np.uint8)
    case.e2 = np.clip(case.e2.astype(int) - rng.integers(-20, 21, size=(1, case.I // 32, 1)), 60, 200).astype(np.uint8)
    check(case)


def test_ties_go_to_the_lower_index():
    """Equal router rows: the lower expert index wins, and its weight is theirs."""
    case = Case(4, 12, 3, 96, 64, seed=6)
    case.router[:] = case.router[0]
    ref = Q.route(np.zeros((4, 12)), 3, True)
    assert ref[0].tolist() == [[0, 1, 2]] * 4
    y, bound = case.reference()
    got = torch_to_f64(run(case))
    assert np.all(np.abs(got - y) <= bound)


def test_tokens_do_not_see_one_another():
    case = Case(20, 16, 4, 256, 96, seed=8)
    dev = case.device()
    full = w4.mxfp4_moe(*dev, 4)
    for t in (0, 7, 19):
        one = w4.mxfp4_moe(dev[0][t:t + 1].contiguous(), *dev[1:], 4)
        assert torch.equal(one[0], full[t])
    bad = dev[0].clone()
    bad[3, 11] = float("nan")
    bad[9] = float("inf")
    y = w4.mxfp4_moe(bad, *dev[1:], 4)
    keep = [t for t in range(20) if t not in (3, 9)]
    assert torch.equal(y[keep], full[keep])
    assert bool(torch.isnan(y[3]).all()) and bool(torch.isnan(y[9]).all())
    zero = dev[0].clone()
    zero[5] = 0
    assert torch.count_nonzero(w4.mxfp4_moe(zero, *dev[1:], 4)[5]) == 0
    assert w4.device_status() == w4.OK


@pytest.mark.parametrize("T,E,k,H,I", [
    (64, 128, 4, 2080, 64),      # many router tiles in one call, few in the other; three stages of K
    (64, 12, 6, 1056, 544),      # several groups per expert, several items per thread block, 3 and 2 stages
    (40, 24, 3, 544, 1056),
])
def test_a_token_alone_and_among_many(T, E, k, H, I):
    """Bit for bit the same, whatever share of the call's work the token is."""
    gen = torch.Generator().manual_seed(T + H)
    rand = lambda *s: torch.randn(*s, generator=gen)
    words = lambda *s: torch.randint(-2 ** 31, 2 ** 31 - 1, s, generator=gen, dtype=torch.int32).cuda()
    scales = lambda *s: torch.randint(118, 122, s, generator=gen, dtype=torch.uint8).cuda()
    x = rand(T, H).bfloat16().cuda()
    rest = ((rand(E, H) / H ** 0.5).bfloat16().cuda(), words(E, H // 8, 2 * I), scales(E, H // 32, 2 * I),
            words(E, I // 8, H), scales(E, I // 32, H), k)
    full = w4.mxfp4_moe(x, *rest, renormalize=False)
    assert bool(torch.isfinite(full).all())
    for first, last in ((0, 1), (T // 2, T // 2 + 1), (T - 1, T), (5, 14), (3, T - 2)):
        assert torch.equal(w4.mxfp4_moe(x[first:last].contiguous(), *rest, renormalize=False), full[first:last])


def test_nan_scale_of_an_expert_stays_with_its_tokens():
    case = Case(12, 6, 2, 128, 64, seed=9)
    ref, bound = case.reference()
    case.e13[4, 1, 5] = 255
    got = torch_to_f64(run(case))
    hit = (Q.route(case.logits(), 2, True)[0] == 4).any(axis=1)
    assert hit.any() and not hit.all()
    assert np.all(np.isnan(got[hit]))
    assert np.all(np.abs(got - ref)[~hit] <= bound[~hit])


def test_workspace_streams_and_graphs():
    """One workspace for shapes in any order, a side stream, and a replayed graph."""
    cases = [Case(*s, seed=11) for s in ((1, 8, 2, 64, 32), (30, 20, 4, 544, 352), (2, 250, 16, 1024, 64))]
    dev = [c.device() for c in cases]
    need = max(w4.load_library().w4a16_mxfp4_moe_workspace_bytes(c.T, c.E, c.k, c.H, c.I) for c in cases)
    ref = [w4.mxfp4_moe(*d, c.k) for d, c in zip(dev, cases)]
    ws = w4.new_workspace(need)
    order = [0, 1, 2, 1, 0, 2, 0]
    for i in order:
        assert torch.equal(w4.mxfp4_moe(*dev[i], cases[i].k, workspace=ws), ref[i])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [w4.mxfp4_moe(*dev[i], cases[i].k, stream=side) for i in order]
    torch.cuda.synchronize()
    for g, i in zip(got, order):
        assert torch.equal(g, ref[i])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [w4.mxfp4_moe(*dev[i], cases[i].k) for i in order]
    for o in outs:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for o, i in zip(outs, order):
        assert torch.equal(o, ref[i])
    assert w4.device_status() == w4.OK


def test_binding_refusals():
    case = Case(2, 4, 2, 64, 32, seed=12)
    x, r, w13, e13, w2, e2 = case.device()
    with pytest.raises(TypeError):
        w4.mxfp4_moe(x.half(), r, w13, e13, w2, e2, 2)
    with pytest.raises(TypeError):
        w4.mxfp4_moe(x, r, w13[0], e13, w2, e2, 2)
    with pytest.raises(ValueError):
        w4.mxfp4_moe(x, r[:3].contiguous(), w13, e13, w2, e2, 2)
    with pytest.raises(ValueError):
        w4.mxfp4_moe(x, r, w13, e13[:, :, :32].contiguous(), w2, e2, 2)
    with pytest.raises(ValueError):
        w4.mxfp4_moe(x.t().contiguous().t(), r, w13, e13, w2, e2, 2)
    for k in (0, 5):
        with pytest.raises(w4.W4A16Error) as err:
            w4.mxfp4_moe(x, r, w13, e13, w2, e2, k)
        assert err.value.status == w4.ERR_SHAPE
    with pytest.raises(w4.W4A16Error) as err:
        w4.mxfp4_moe(torch.zeros((65, 64), dtype=torch.bfloat16, device="cuda"), r, w13, e13, w2, e2, 2)
    assert err.value.status == w4.ERR_SHAPE
    with pytest.raises(w4.W4A16Error) as err:
        w4.mxfp4_moe(x, r, w13, e13, w2, e2, 2, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    assert err.value.status == w4.ERR_WORKSPACE
