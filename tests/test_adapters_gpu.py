"""The adapters by token, forward and backward, against their definitions in binary64.

Tolerances, derived from the arithmetic (u = 2^-24; bf16 rounds by at most 2^-8 relative):
 - u and du are binary32 sums of exact products (du of binary32 sums, times the scale): a sum of n products, added 8 or
   more at a time and in 8 or fewer waves and 16 or fewer ranges, is off by at most (n / 8 + 32) u of the sum of magnitudes;
 - u (times the scale, one rounding) enters its second product as two bf16 parts, which leave 2^-16 of it; that product
   adds its terms in binary32 likewise (over r, or over the tokens of a piece and then the pieces);
 - outputs in bf16 are rounded once.
Every bound is evaluated entry by entry from the inputs; products of two roundings are covered by a factor 1 + 2^-6.
"""
import pytest
import torch

from bit_quantized_lora_02_amd import binding as B
from bit_quantized_lora_02_amd.synth import linear_inputs
from test_step_gpu import BF, Guarded, U, bf, check

pytestmark = pytest.mark.gpu
PART = 2.0 ** -16


def depth(n):
    return (n / 8 + 32) * U


def make(T, K, N, pool, r, kind, ranks, seed):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, dtype=torch.float32)  # noqa: E731
    if kind == "one":
        index = torch.full((T,), pool - 1)
    elif kind == "none":
        index = torch.tensor([-1, pool, -(1 << 31), (1 << 31) - 1])[torch.randint(0, 4, (T,), generator=g)]
    else:
        index = torch.randint(0, pool, (T,), generator=g)
        if kind == "runs":  # sequences of one adapter each, the last one short
            index = index.repeat_interleave(max(1, T // 5))[:T]
        none = torch.rand(T, generator=g) < 0.15
        index = torch.where(none, torch.tensor([-1, pool, pool + 7])[torch.randint(0, 3, (T,), generator=g)], index)
    rank = None
    if ranks:
        rank = torch.randint(0, r + 1, (pool,), generator=g)
        rank[0] = r
        if pool > 2:
            rank[1], rank[2] = 0, min(5, r)
    X, dY = rn(T, K).to(bf), rn(T, N).to(bf)
    A, Bp = (rn(pool, r, K) / K ** 0.5).to(bf), rn(pool, N, r).to(bf)
    scale = 0.25 + 2 * torch.rand(pool, generator=g)
    return dict(X=X, dY=dY, A=A, B=Bp, scale=scale, index=index.to(torch.int32), rank=None if rank is None else rank.int(),
                base=rn(T, N).to(bf), dbase=rn(T, K).to(bf))


def spoil(s):
    """NaN wherever nothing may be read: rows of X and dY without an adapter, what lies past the ranks."""
    pool, r = s["A"].shape[:2]
    none = (s["index"] < 0) | (s["index"] >= pool)
    s["X"][none] = float("nan")
    s["dY"][none] = float("nan")
    if s["rank"] is not None:
        past = torch.arange(r)[None, :] >= s["rank"][:, None]
        s["A"][past] = float("nan")
        s["B"].transpose(1, 2)[past] = float("nan")


def reference(s, dev="cpu"):
    """(Y, U, dX, dA, dB) and their bounds in binary64; U is what the backward takes for u (binary32 of the exact one)."""
    X, dY, A, Bp, scale = (s[k].to(dev).double() for k in ("X", "dY", "A", "B", "scale"))
    (T, K), (pool, N, r) = X.shape, Bp.shape
    z = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device=dev)  # noqa: E731
    Y, dX, u_all, dA, dB = s["base"].to(dev).double(), s["dbase"].to(dev).double(), z(T, r), z(pool, r, K), z(pool, N, r)
    bY, bX, bU, bA, bB = (z(*t.shape) for t in (Y, dX, u_all, dA, dB))
    for a in range(pool):
        t = (s["index"] == a).nonzero()[:, 0].to(dev)
        k = r if s["rank"] is None else int(s["rank"][a])
        n = len(t)
        if not n or not k:
            continue
        x, g, Aa, Ba, sc = X[t], dY[t], A[a, :k], Bp[a, :, :k], float(scale[a])
        At, Bt = Aa.t().contiguous(), Ba.t().contiguous()
        u, e_u = x @ At, depth(K) * (x.abs() @ At.abs())
        u_all[t, :k], bU[t, :k] = u, e_u
        Y[t] += sc * (u @ Bt)
        bY[t] = sc * ((e_u + (PART + U) * u.abs() + depth(r) * u.abs()) @ Bt.abs())
        du, e_du = sc * (g @ Ba), sc * depth(N) * (g.abs() @ Ba.abs())
        dX[t] += du @ Aa
        bX[t] = (e_du + (PART + U + depth(r)) * du.abs()) @ Aa.abs()
        dA[a, :k] = du.t().contiguous() @ x
        bA[a, :k] = (e_du + (PART + U + depth(n)) * du.abs()).t().contiguous() @ x.abs()
        u32 = u.float().double()
        dB[a, :, :k] = sc * (g.t().contiguous() @ u32)
        bB[a, :, :k] = sc * (g.abs().t().contiguous() @ ((PART + U + depth(n)) * u32.abs()))
        # (U recomputed is e_u off what is given here: the bound of dB without U)
        s.setdefault("e_dB", z(pool, N, r))[a, :, :k] = sc * (g.abs().t().contiguous() @ e_u)
    for y, b in ((Y, bY), (dX, bX), (dA, bA), (dB, bB)):
        b += (BF + U) * y.abs()
    return (Y, u_all, dX, dA, dB), (bY, bU, bX, bA, bB)


SIZES = [  # T, n_in, n_out, pool, r, tokens, ranks
    (1, 8, 8, 1, 8, "any", False), (1, 4096, 512, 64, 16, "any", False), (5, 264, 1000, 3, 8, "any", True),
    (16, 2048, 264, 64, 16, "any", False), (33, 520, 72, 4, 32, "runs", True), (64, 1032, 2056, 1000, 24, "any", True),
    (64, 512, 512, 2, 64, "one", False), (65, 512, 264, 3, 16, "any", True), (65, 72, 8, 1000, 128, "any", False),
    (100, 4104, 136, 5, 128, "runs", True), (129, 200, 200, 7, 40, "none", False), (300, 1000, 776, 9, 48, "any", True),
    (777, 4096, 2048, 6, 16, "runs", True), (1500, 520, 520, 2, 72, "one", True), (2048, 264, 1032, 8, 32, "runs", False),
    (2500, 776, 264, 12, 128, "any", True), (5000, 136, 72, 100, 16, "any", True), (9001, 72, 264, 3, 8, "runs", False),
    (20000, 8, 16, 17, 8, "any", True)]


@pytest.mark.parametrize("T,K,N,pool,r,kind,ranks", SIZES)
def test_adapters(T, K, N, pool, r, kind, ranks):
    print(f"adapters T={T} {K}x{N} pool={pool} r={r} {kind} ranks={ranks}", flush=True)
    s = make(T, K, N, pool, r, kind, ranks, T + K)
    dev = "cuda" if T * K * N * r > 1 << 34 else "cpu"
    clean = dict(s, **{k: s[k].clone() for k in ("X", "dY", "A", "B")})
    spoil(s)
    for k in ("X", "dY", "A", "B"):
        clean[k] = torch.where(torch.isnan(s[k]), torch.zeros(1, dtype=bf), s[k])
    (Y, u, dX, dA, dB), (bY, bU, bX, bA, bB) = reference(clean, dev)
    g = {k: None if s[k] is None else s[k].cuda() for k in ("X", "dY", "A", "B", "scale", "index", "rank", "base", "dbase")}
    pools = (g["A"], g["B"], g["scale"], g["index"], g["rank"])
    none = ((s["index"] < 0) | (s["index"] >= pool)).to(dev)
    for base in (g["base"], None):
        out, u_out = Guarded(torch.full((T, N), float("nan"), dtype=bf)), Guarded(torch.full((T, r), float("nan")))
        ws = Guarded(torch.full((B.adapters_workspace_bytes(T, K, N, pool, r),), 0x5A, dtype=torch.uint8))
        got, got_u = B.adapters_fwd(g["X"], *pools, base=base, out=out.t, u_out=u_out.t, ws=ws.t)
        torch.cuda.synchronize()
        assert out.intact() and u_out.intact() and ws.intact()
        want = Y if base is not None else Y - s["base"].to(dev).double()
        check("Y", got, want, bY + (0 if base is not None else BF * want.abs()))
        check("U", got_u, u, bU)
        assert (got_u.to(dev)[none] == 0).all()
        if base is not None:
            assert torch.equal(got.to(dev)[none], base.to(dev)[none])
    again, nothing = B.adapters_fwd(g["X"], *pools, base=g["base"], save_u=False)
    assert nothing is None
    in_place = g["base"].clone()
    B.adapters_fwd(g["X"], *pools, base=in_place, out=in_place)
    assert torch.equal(in_place, again), "not repeatable, or Y over base differs"
    U32 = u.float().cuda()
    U32[none.cuda()] = float("nan")  # not read
    for U_in, base, need in ((U32, g["dbase"], (True, True, True)), (None, g["dbase"], (True, True, True)),
                             (U32, None, (True, False, False)), (U32, g["dbase"], (False, True, False)),
                             (U32, g["dbase"], (False, False, True)), (None, None, (False, True, True))):
        outs = [Guarded(torch.full(t.shape, float("nan"), dtype=bf)) for t in (s["X"], s["A"], s["B"])]
        ws = Guarded(torch.full((B.adapters_workspace_bytes(T, K, N, pool, r, True),), 0x5A, dtype=torch.uint8))
        got = B.adapters_bwd(g["X"], g["dY"], *pools, U=U_in, base=base, ws=ws.t,
                             outs=tuple(o.t if n else None for o, n in zip(outs, need)))
        torch.cuda.synchronize()
        assert all(o.intact() for o in outs) and ws.intact()
        assert [x is not None for x in got] == list(need)
        if need[0]:
            want = dX if base is not None else dX - s["dbase"].to(dev).double()
            check("dX", got[0], want, bX + (0 if base is not None else BF * want.abs()))
        if need[1]:
            check("dA", got[1], dA, bA)
        if need[2]:
            check("dB", got[2], dB, bB + (clean["e_dB"] if U_in is None and "e_dB" in clean else 0))
        if need[1] and need[2] and ranks:
            past = (torch.arange(r)[None, :] >= s["rank"][:, None]).cuda()
            assert (got[1][past] == 0).all() and (got[2].transpose(1, 2)[past] == 0).all()
        if all(need):
            in_place = g["dbase"].clone()
            same = B.adapters_bwd(g["X"], g["dY"], *pools, U=U_in, base=in_place, outs=(in_place, outs[1].t.clone(),
                                                                                        outs[2].t.clone()))
            assert all(torch.equal(p, q) for p, q in zip(same, got)), "not repeatable, or dX over base differs"


def test_no_tokens():
    s = make(4, 64, 72, 3, 8, "any", False, 1)
    g = {k: s[k].cuda() for k in ("A", "B", "scale")}
    X, dY = torch.zeros(0, 64, dtype=bf, device="cuda"), torch.zeros(0, 72, dtype=bf, device="cuda")
    index = torch.zeros(0, dtype=torch.int32, device="cuda")
    Y, u = B.adapters_fwd(X, g["A"], g["B"], g["scale"], index)
    assert Y.shape == (0, 72) and u.shape == (0, 8)
    dX, dA, dB = B.adapters_bwd(X, dY, g["A"], g["B"], g["scale"], index)
    assert dX.shape == (0, 64) and (dA == 0).all() and (dB == 0).all()


def test_ranks_out_of_range_are_cut():
    s = make(70, 64, 72, 3, 16, "any", False, 2)
    g = [s[k].cuda() for k in ("X", "A", "B", "scale", "index")]
    want = B.adapters_fwd(*g, rank=torch.tensor([16, 0, 16], dtype=torch.int32, device="cuda"))
    got = B.adapters_fwd(*g, rank=torch.tensor([99, -4, 1 << 30], dtype=torch.int32, device="cuda"))
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_as_the_segment_form():
    """With one adapter per segment, one rank and scale, the sum of the NF4 projection and the adapters is
    linear_fwd_multi's, whose u has one more rounding to bf16."""
    T, K, N, r, pool, alpha = 200, 256, 264, 16, 3, 16.0
    inp = linear_inputs(N, K, T, r, alpha, seed=4)
    w = B.quantize_nf4(torch.from_numpy(inp.W).cuda())
    s = make(T, K, N, pool, r, "any", False, 3)
    X, A, Bp = s["X"].cuda(), s["A"].cuda(), s["B"].cuda()
    seg = torch.tensor([0, 70, 70, 150, T], dtype=torch.int32, device="cuda")
    ad = torch.tensor([2, 0, -1, 1], dtype=torch.int32, device="cuda")
    Y = B.linear_fwd_multi(X, w, A, Bp, alpha, seg, ad)
    index = torch.cat([torch.full((70,), 2), torch.full((80,), -1), torch.full((50,), 1)]).int().cuda()
    shared = B.linear_fwd_multi(X, w, A, Bp, alpha, seg, torch.full_like(ad, -1))
    got, u = B.adapters_fwd(X, A, Bp, torch.full((pool,), alpha / r, device="cuda"), index, base=shared)
    terms = torch.zeros(T, N, dtype=torch.float64, device="cuda")
    for a in (1, 2):
        t = index == a
        terms[t] = u[t].double().abs() @ Bp[a].double().abs().t().contiguous()
    bound = 3 * BF * (got.double().abs() + shared.double().abs()) + BF * alpha / r * terms
    assert ((got.double() - Y.double()).abs() <= bound + 1e-6).all()


def test_gradients_against_differences():
    """The gradients against central differences of the definition in binary64 (bilinear: no error of second order)."""
    s = make(90, 72, 136, 4, 24, "any", True, 6)
    g = torch.Generator().manual_seed(1)
    rank = s["rank"]
    mine = torch.nn.functional.one_hot(s["index"].long().clamp(-1, 4) % 5, 5)[:, :4].double()

    def f(X, A, Bp):
        on = (torch.arange(24)[None, :] < rank[:, None]).double()
        u = torch.einsum("tk,ajk->taj", X, A) * on * mine[:, :, None]
        return (s["dY"].double() * torch.einsum("taj,anj->tn", u * s["scale"].double()[:, None], Bp)).sum()

    c = {k: v.cuda() for k, v in s.items()}
    grads = B.adapters_bwd(c["X"], c["dY"], c["A"], c["B"], c["scale"], c["index"], rank=c["rank"])
    at = [s[k].double() for k in ("X", "A", "B")]
    for i, grad in enumerate(grads):
        v = torch.randn(at[i].shape, generator=g, dtype=torch.float64)
        plus, minus = ([a + (0.5 * sign * v if j == i else 0) for j, a in enumerate(at)] for sign in (1, -1))
        slope = float(f(*plus) - f(*minus))
        terms = grad.double().cpu() * v
        assert abs(float(terms.sum()) - slope) <= (BF + 2 * PART) * float(terms.abs().sum()) + 1e-6


def test_step_of_many_adapters():
    """A step as a user runs it: embedding, norm, the NF4 projection with its own adapter and the requests' adapters beside
    it, norm, cross entropy, and back to every trained tensor; gradients against torch's of the same graph in binary64."""
    torch.manual_seed(0)
    T, K, V, r, pool = 150, 256, 500, 16, 4
    inp = linear_inputs(K, K, T, r, 16.0, seed=1)
    w = B.quantize_nf4(torch.from_numpy(inp.W).cuda())
    s = make(T, K, K, pool, r, "any", True, 8)
    rnd = lambda *shape, std=1.0: (torch.randn(*shape, device="cuda") * std)  # noqa: E731
    leaves = dict(E=rnd(V, K).to(bf), g1=1 + rnd(K, std=0.1), b1=rnd(K, std=0.1), A=rnd(r, K, std=0.05).to(bf),
                  B=rnd(K, r, std=0.05).to(bf), Ap=s["A"].cuda(), Bp=(s["B"] * 0.1).cuda(), g2=(1 + rnd(K, std=0.1)).to(bf),
                  H=rnd(V, K, std=0.06).to(bf))
    for t in leaves.values():
        t.requires_grad_(True)
    tokens, labels = torch.randint(0, V, (T,), device="cuda"), torch.randint(0, V, (T,), device="cuda")
    scale, index, rank = s["scale"].cuda(), s["index"].cuda(), s["rank"].cuda()
    weight = torch.full((T,), 1.0 / 128, device="cuda")
    x = B.LayerNormFn.apply(B.EmbedFn.apply(tokens, leaves["E"], 4.0), leaves["g1"], leaves["b1"])
    shared = B.QLoRALinearFn.apply(x, w, leaves["A"], leaves["B"], 16.0)
    y = B.AdaptersFn.apply(x, leaves["Ap"], leaves["Bp"], scale, index, rank, shared)
    total, _ = B.HeadCEFn.apply(B.LayerNormFn.apply(y, leaves["g2"]), leaves["H"], labels, weight)
    total.backward()

    ref = {k: t.detach().double().cpu().requires_grad_(True) for k, t in leaves.items()}
    norm = torch.nn.functional.layer_norm
    x = norm(ref["E"][tokens.cpu()] * 4.0, (K,), ref["g1"], ref["b1"], 1e-5)
    W = B.dequant(w).double().cpu()
    on = (torch.arange(r)[None, :] < s["rank"][:, None]).double()
    mine = torch.nn.functional.one_hot(torch.where((s["index"] >= 0) & (s["index"] < pool), s["index"], pool).long(), pool + 1)
    u = torch.einsum("tk,ajk->taj", x, ref["Ap"]) * on * mine[:, :pool, None].double()
    y = x @ W.t() + (x @ ref["A"].t()) @ ref["B"].t() + torch.einsum("taj,anj->tn", u * s["scale"].double()[:, None], ref["Bp"])
    z = norm(y, (K,), ref["g2"], None, 1e-5) @ ref["H"].t()
    want = torch.nn.functional.cross_entropy(z, labels.cpu(), reduction="sum") / 128
    want.backward()
    assert abs(total.item() - want.item()) <= 2 * BF * abs(want.item())
    for k, t in leaves.items():
        # every activation and gradient between the calls is rounded to bf16 once (six of them on the way back from the
        # loss to the embedding, as many on the way there): their errors add as a random sum, well under 16 roundings
        rel = float((t.grad.double().cpu() - ref[k].grad).norm() / ref[k].grad.norm())
        assert rel <= 16 * BF, f"{k}: {rel:.2e}"


def test_streams_layouts_and_overlapping_calls():
    s = make(300, 264, 520, 5, 16, "any", True, 11)
    c = {k: v.cuda() for k, v in s.items()}
    call = lambda X, A: (*B.adapters_fwd(X, A, c["B"], c["scale"], c["index"], rank=c["rank"], base=c["base"]),  # noqa: E731
                         *B.adapters_bwd(X, c["dY"], A, c["B"], c["scale"], c["index"], rank=c["rank"]))
    want = call(c["X"], c["A"])
    wide = torch.empty(300, 528, dtype=bf, device="cuda")
    wide[:, ::2] = c["X"]
    A_t = c["A"].transpose(1, 2).contiguous().transpose(1, 2)
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for st in streams:  # calls that overlap in time, each with its own workspace
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            got.append(call(wide[:, ::2], A_t))
    torch.cuda.synchronize()
    for results in got:
        assert all(torch.equal(p, q) for p, q in zip(results, want))


@pytest.mark.parametrize("T", [48, 700])
def test_graph_replays(T):
    """Captured forward and backward replayed on new inputs, other adapters among them, with eager work between."""
    s = make(T, 264, 520, 6, 32, "any", False, 12)
    c = {k: v.cuda() for k, v in s.items() if v is not None}
    rank = torch.full((6,), 32, dtype=torch.int32, device="cuda")

    def step():
        Y, u = B.adapters_fwd(c["X"], c["A"], c["B"], c["scale"], c["index"], rank=rank, base=c["base"])
        return (Y, u, *B.adapters_bwd(c["X"], c["dY"], c["A"], c["B"], c["scale"], c["index"], rank=rank, U=u, base=c["dbase"]))

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        c["X"].normal_()
        c["index"].random_(-1, 6)
        rank.random_(0, 33)
        graph.replay()
        got = [t.clone() for t in out]
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, step())), f"replay {i}"


def test_rows_beyond_four_gib():
    """Offsets past 2^32 bytes of Y, dY, X and dX: rows at the ends against a call on those rows alone."""
    T, N, K, r = 66000, 32776, 64, 8
    g = torch.Generator(device="cuda").manual_seed(0)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda").to(bf)  # noqa: E731
    X, A, Bp = rn(T, K), rn(2, r, K), rn(2, N, r)
    scale = torch.tensor([0.5, 2.0], device="cuda")
    index = (torch.arange(T, device="cuda", dtype=torch.int32) // 7) % 3 - 1
    at = torch.tensor([0, 1, 65000, 65534, 65535, 65536, T - 9, T - 1], device="cuda")
    Y, u = B.adapters_fwd(X, A, Bp, scale, index)
    few, u_few = B.adapters_fwd(X[at], A, Bp, scale, index[at])
    assert torch.equal(u[at], u_few) and torch.equal(Y[at], few)
    dX, dA, dB = B.adapters_bwd(X, Y, A, Bp, scale, index, U=u)
    few = B.adapters_bwd(X[at], Y[at].contiguous(), A, Bp, scale, index[at])[0]
    # (both round dX once, each by at most BF of it; du of few tokens is added from ranges of n_out, binary32 sums in
    # another order, which move dX by less than a tenth of that)
    rel = float((dX[at].double() - few.double()).norm() / few.double().norm())
    assert rel <= 2.1 * BF and torch.isfinite(dA.float()).all() and torch.isfinite(dB.float()).all()
    # the same adapters the other way round: the wide side is the input
    del dX, dA, dB
    A2, B2 = rn(2, r, N), rn(2, K, r)
    Z, v = B.adapters_fwd(Y, A2, B2, scale, index)
    few, v_few = B.adapters_fwd(Y[at].contiguous(), A2, B2, scale, index[at])
    assert float((v[at].double() - v_few.double()).norm() / v_few.double().norm()) <= depth(N) and Z.shape == (T, K)
    dX = B.adapters_bwd(Y, Z, A2, B2, scale, index, U=v, need_dw=False)[0]
    few = B.adapters_bwd(torch.zeros(len(at), N, dtype=bf, device="cuda"), Z[at], A2, B2, scale, index[at])[0]
    assert torch.equal(dX[at], few)


def test_pools_of_many_blocks():
    """Pools that are transposed in more blocks than one launch has workgroups."""
    T, K, N, pool, r = 200, 8192, 8192, 1000, 8
    assert pool * (K + N) // 1024 > 8192
    s = make(T, K, N, pool, r, "any", False, 3)
    want, bounds = reference(s, "cuda")
    g = {k: s[k].cuda() for k in ("X", "dY", "A", "B", "scale", "index", "dbase")}
    got = B.adapters_bwd(g["X"], g["dY"], g["A"], g["B"], g["scale"], g["index"], U=want[1].float(), base=g["dbase"])
    for name, x, y, b in zip(("dX", "dA", "dB"), got, want[2:], bounds[2:]):
        check(name, x, y, b)


@pytest.mark.parametrize("T,pool,kind", [(8192, 5, "any"), (8193, 1000, "any"), (40000, 1000, "any"), (70001, 3, "runs")])
def test_many_tokens(T, pool, kind):
    """Tokens that one workgroup, and several, bring into groups."""
    test_adapters(T, 16, 8, pool, 8, kind, True)


@pytest.mark.parametrize("T,N,r,off", [(1500, 12008, 16, 0), (2500, 8072, 40, 0), (2100, 16200, 24, 0), (2100, 16384, 128, 8),
                                       (3000, 6008, 72, 24), (1200, 14400, 8, 40)])
def test_large_outputs_of_odd_widths(T, N, r, off):
    """Outputs past the caches whose rows do not begin with a line of memory, with and without a base, and over it."""
    print(f"adapters T={T} N={N} r={r} output {2 * off} bytes off a line", flush=True)
    K = 72
    s = make(T, K, N, 3, r, "any", True, N + r)
    want, bounds = reference(s, "cuda")
    g = {k: s[k].cuda() for k in ("X", "dY", "A", "B", "scale", "index", "rank", "base")}
    pools = (g["A"], g["B"], g["scale"], g["index"], g["rank"])
    plain = want[0] - g["base"].double()
    for base in (None, g["base"]):
        whole = torch.full((off + T * N + 64,), 7.0, dtype=bf, device="cuda")
        out = whole[off:off + T * N].view(T, N)
        B.adapters_fwd(g["X"], *pools, base=base, out=out)
        torch.cuda.synchronize()
        assert (whole[:off] == 7).all() and (whole[off + T * N:] == 7).all()
        check("Y", out, plain if base is None else want[0], bounds[0] + (BF * plain.abs() if base is None else 0))
    whole[off:off + T * N] = g["base"].view(-1)
    B.adapters_fwd(g["X"], *pools, base=out, out=out)
    check("Y over base", out, want[0], bounds[0])
    # the same as dX, whose wide side is n_in
    s2 = make(T, N, K, 3, r, "runs", True, N)
    want, bounds = reference(s2, "cuda")
    g = {k: s2[k].cuda() for k in ("X", "dY", "A", "B", "scale", "index", "rank", "dbase")}
    got = B.adapters_bwd(g["X"], g["dY"], g["A"], g["B"], g["scale"], g["index"], g["rank"], U=want[1].float(), base=g["dbase"])
    for name, x, y, b in zip(("dX", "dA", "dB"), got, want[2:], bounds[2:]):
        check(name, x, y, b)


@pytest.mark.parametrize("T", [90, 700, 2100])
@pytest.mark.parametrize("r", range(8, 129, 8))
def test_every_rank(T, r):
    test_adapters(T, 328, 264, 3, r, "any", True)


@pytest.mark.parametrize("T,r", [(0, 16), (40, 24), (100, 128), (700, 72), (2500, 16)])
def test_scales_of_adapters_without_tokens(T, r):
    """An adapter that no token names has gradients of zeros, whatever its scale holds."""
    print(f"adapters T={T} r={r}, scales that are not finite", flush=True)
    pool, K, N = 5, 72, 136
    s = make(T, K, N, pool, r, "any", False, T + r)
    s["index"] = torch.tensor([1, 3, -1], dtype=torch.int32)[torch.arange(T) % 3]
    g = {k: v.cuda() for k, v in s.items() if v is not None}
    call = lambda scale: B.adapters_bwd(g["X"], g["dY"], g["A"], g["B"], scale, g["index"])  # noqa: E731
    want = call(g["scale"])
    odd = g["scale"].clone()
    odd[0], odd[2], odd[4] = float("nan"), float("inf"), float("-inf")
    got = call(odd)
    for name, x, y in zip(("dX", "dA", "dB"), got, want):
        assert torch.equal(x, y), name
    for a in range(pool):
        if T == 0 or a not in (1, 3):
            assert (got[1][a] == 0).all() and (got[2][a] == 0).all()


def kinds(t):
    """0: finite, 1: +inf, 2: -inf, 3: NaN."""
    t = t.double().cpu()
    return torch.isposinf(t) * 1 + torch.isneginf(t) * 2 + torch.isnan(t) * 3


@pytest.mark.parametrize("T,r", [(40, 8), (60, 72), (100, 16), (128, 128), (300, 40), (700, 16), (900, 120), (2500, 32), (2600, 104)])
def test_infinities(T, r):
    """An infinite u or du gives what the formulas give: infinities, NaN where both signs meet, in that token's rows and
    that adapter's gradients alone.  The tokens are the last of their groups, behind which a tile has more places."""
    print(f"adapters T={T} r={r} infinite", flush=True)
    pool, K, N = 4, 72, 136
    s = make(T, K, N, pool, r, "any", False, T + r)
    s["A"][:, :, ::2] = s["A"][:, :, ::2].abs() + 0.125
    s["B"][:, ::2] = s["B"][:, ::2].abs() + 0.125
    last = [int((s["index"] == a).nonzero()[-1]) for a in range(pool)]
    g = {k: v.cuda() for k, v in s.items() if v is not None}
    pools = (g["A"], g["B"], g["scale"], g["index"])
    A, Bp = s["A"].double(), s["B"].double()
    inf = float("inf")

    # X of two tokens: u, Y and, with u formed again, dB
    X, clean = g["X"].clone(), g["X"].clone()
    for a, value in ((1, inf), (2, -inf), (3, float("nan"))):
        X[last[a], 4], clean[last[a]] = value, 0
    Y, u = B.adapters_fwd(X, *pools, base=g["base"])
    want_Y, want_u = (t.clone() for t in B.adapters_fwd(clean, *pools, base=g["base"]))
    dB = B.adapters_bwd(X, g["dY"], *pools, outs=(None, None, torch.empty_like(g["B"])))[2]
    want_dB = B.adapters_bwd(clean, g["dY"], *pools, outs=(None, None, torch.empty_like(g["B"])))[2]
    for a in (1, 2, 3):
        t = last[a]
        u_t = X[t].double().cpu() @ A[a].t().contiguous()
        assert (kinds(u_t) == a).all() and torch.equal(kinds(u[t]), kinds(u_t))
        assert torch.equal(kinds(Y[t]), kinds(u_t @ Bp[a].t().contiguous())), f"Y of an infinite u, adapter {a}"
        assert (kinds(Y[t])[::2] == a).all()
        assert torch.equal(kinds(dB[a]), kinds(s["dY"][t].double()[:, None] * u_t)), f"dB of an infinite u, adapter {a}"
        Y[t], u[t], dB[a] = want_Y[t], want_u[t], want_dB[a]
    assert torch.equal(Y, want_Y) and torch.equal(u, want_u) and torch.equal(dB, want_dB)

    # dY of a token: du, dX and dA; a given u: dB
    dY, clean = g["dY"].clone(), g["dY"].clone()
    dY[last[0], 6], clean[last[0]] = -inf, 0
    U, clean_U = want_u.clone(), want_u.clone()
    U[last[3]], clean_U[last[3]] = inf, 0
    got = B.adapters_bwd(g["X"], dY, *pools, U=U, base=g["dbase"])
    want = B.adapters_bwd(g["X"], clean, *pools, U=clean_U, base=g["dbase"])
    t = last[0]
    du = dY[t].double().cpu() @ Bp[0]
    assert torch.isneginf(du).all()
    assert torch.equal(kinds(got[0][t]), kinds(du @ A[0])), "dX of an infinite du"
    assert (kinds(got[0][t])[::2] == 2).all()
    assert torch.equal(kinds(got[1][0]), kinds(du[:, None] * s["X"][t].double())), "dA of an infinite du"
    t3 = last[3]
    assert torch.equal(kinds(got[2][3]), kinds((s["dY"][t3].double() * inf)[:, None].expand(N, r))), "dB of an infinite u"
    got[0][t], got[1][0], got[2][3], got[2][0] = want[0][t], want[1][0], want[2][3], want[2][0]
    for name, x, y in zip(("dX", "dA", "dB"), got, want):
        assert torch.equal(x, y), name


@pytest.mark.parametrize("T", [3, 200, 2100])
def test_largest_values(T):
    """u finite and past bf16's range: 2^128 - 2^118, cancelled by the base to what its low part alone gives."""
    K, N, r = 72, 264, 8
    X = torch.zeros(T, K, dtype=bf, device="cuda")
    X[:, 0], X[:, 1] = 2.0 ** 127 * (2 - 2.0 ** -7), 0.75 * 2.0 ** 120
    A = torch.zeros(1, r, K, dtype=bf, device="cuda")
    A[:, :, :2] = 1
    Bp = torch.full((1, N, r), 2.0 ** -100, dtype=bf, device="cuda")
    base = torch.full((T, N), -8 * 2.0 ** 27 * (2 - 2.0 ** -7), dtype=bf, device="cuda")
    scale, index = torch.ones(1, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
    Y, u = B.adapters_fwd(X, A, Bp, scale, index, base=base)
    assert (u.double() == 2.0 ** 128 - 2.0 ** 118).all()
    assert (Y == 6 * 2.0 ** 20).all()


@pytest.mark.parametrize("T,r,rank", [(20, 8, 8), (200, 24, 24), (2100, 40, 3)])
def test_infinite_scale(T, r, rank):
    """What lies past the rank takes no part in a product with an infinite scale either."""
    K, N = 72, 136
    s = make(T, K, N, 2, r, "any", False, T)
    g = {k: v.cuda() for k, v in s.items() if v is not None}
    X, A, Bp = (g[k].abs() for k in ("X", "A", "B"))
    ranks = torch.full((2,), rank, dtype=torch.int32, device="cuda")
    want, _ = B.adapters_fwd(X, A, Bp, g["scale"], g["index"], rank=ranks, base=g["base"])
    g["scale"][1] = float("inf")
    Y, _ = B.adapters_fwd(X, A, Bp, g["scale"], g["index"], rank=ranks, base=g["base"])
    mine = g["index"] == 1
    assert torch.isposinf(Y[mine]).all() and torch.equal(Y[~mine], want[~mine])


@pytest.mark.parametrize("T,r,ranks", [(90, 24, True), (700, 72, True), (2500, 16, False)])
def test_gradients_entry_by_entry(T, r, ranks):
    """The gradients against torch's of the definition in binary64, u formed again by the backward."""
    K, N, pool = 72, 136, 4
    s = make(T, K, N, pool, r, "any", ranks, T + r)
    leaves = {k: s[k].double().requires_grad_(True) for k in ("X", "A", "B")}
    rank = s["rank"] if ranks else torch.full((pool,), r)
    Y = s["base"].double()
    for a in range(pool):
        t, k = (s["index"] == a).nonzero()[:, 0], int(rank[a])
        u = leaves["X"][t] @ leaves["A"][a, :k].t()
        Y = Y.index_add(0, t, s["scale"][a].double() * (u @ leaves["B"][a, :, :k].t()))
    Y.backward(s["dY"].double())
    bounds = reference(s)[1]
    g = {k: None if v is None else v.cuda() for k, v in s.items() if k != "e_dB"}
    got = B.adapters_bwd(g["X"], g["dY"], g["A"], g["B"], g["scale"], g["index"], g["rank"], base=g["dbase"])
    check("dX", got[0], leaves["X"].grad + s["dbase"].double(), bounds[2])
    check("dA", got[1], leaves["A"].grad, bounds[3])
    # (the bound of dB is that of a given u, rounded from the exact one, and what a recomputed one is off it)
    check("dB", got[2], leaves["B"].grad, bounds[4] + 1.01 * s["e_dB"])


@pytest.mark.parametrize("T", [48, 700])
def test_function_captured(T):
    """Forward and backward of AdaptersFn in one graph, replayed on new inputs with eager work between."""
    s = make(T, 264, 520, 6, 32, "any", True, 12)
    c = {k: v.cuda() for k, v in s.items() if v is not None}
    leaves = [c[k].requires_grad_(True) for k in ("X", "A", "B", "base")]

    def step(X, A, Bp, base):
        Y = B.AdaptersFn.apply(X, A, Bp, c["scale"], c["index"], c["rank"], base)
        return (Y.detach(), *torch.autograd.grad(Y, (X, A, Bp, base), c["dY"]))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*leaves)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*leaves)
    for i in range(4):
        with torch.no_grad():
            for t in (c["dY"], *leaves):
                t.normal_()
        c["index"].random_(-1, 6)
        c["rank"].random_(0, 33)
        want = step(*(t.detach().clone().requires_grad_(True) for t in leaves))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name, p, q in zip(("Y", "dX", "dA", "dB", "dbase"), out, want):
            assert torch.equal(p, q), f"{name} of replay {i}"
