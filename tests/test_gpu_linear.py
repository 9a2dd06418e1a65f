"""Linear attention with a decay for each head against the recurrence in 64 bits: forward, backward, token by token.

Tolerances are those of ``parity.py``: fp32 1e-5 * RMS; bf16 outputs 2e-3 * RMS before their rounding.  The fp32 states
of bf16 inputs are held to 1e-5 * RMS too: their operands are split into parts that keep 24 bits, and an element sums at
most a few thousand products whose errors of 2^-23 each are independent."""
import pytest
import torch

import gated_delta_rule_50_gb300 as gdn
from parity import BF16_TOL, FP32_TOL, check

pytestmark = pytest.mark.gpu
bf16, f32, f64 = torch.bfloat16, torch.float32, torch.float64


def make(B, T, Hq, Hv, K, V, dtype, seed=0, h0=True, packed=False):
    """Inputs on the GPU; packed: q, k and v of a token side by side."""
    gen = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen)

    nq = Hq * K
    if packed:
        side = normal(B, T, 2 * nq + Hv * V).to(dtype).cuda()
        q, k = side[..., :nq].view(B, T, Hq, K), side[..., nq:2 * nq].view(B, T, Hq, K)
        v = side[..., 2 * nq:].view(B, T, Hv, V)
    else:
        q, k, v = (normal(B, T, *s).to(dtype).cuda() for s in ((Hq, K), (Hq, K), (Hv, V)))
    g = -torch.exp2(-8 * torch.rand(Hv, generator=gen))
    g[0] = 0.0
    x = dict(q=q, k=k, v=v, g=g.cuda(), scale=K ** -0.5, h0=None, dht=None)
    x["do"] = normal(B, T, Hv, V).to(dtype).cuda()
    if h0:
        x["h0"], x["dht"] = normal(B, Hv, K, V).cuda(), normal(B, Hv, K, V).cuda()
    return x


def reference(x, spans=None, backward=False):
    """The recurrence token by token in 64 bits; spans: [(row, first, last + 1)] for each state (default: whole rows)."""
    q, k, v, do = (x[n].to(f64) for n in ("q", "k", "v", "do"))
    G = v.shape[2] // q.shape[2]
    q, k = q.repeat_interleave(G, 2), k.repeat_interleave(G, 2)
    B, T, Hv, V = v.shape
    K = q.shape[3]
    spans = spans or [(b, 0, T) for b in range(B)]
    decay = torch.exp(torch.zeros(Hv, device="cuda") if x["g"] is None else x["g"]).to(f64)[:, None, None]
    if x["g"] is not None:
        decay = torch.exp(x["g"].to(f64))[:, None, None]
    zero = torch.zeros(len(spans), Hv, K, V, dtype=f64, device="cuda")
    h0 = zero if x["h0"] is None else x["h0"].to(f64)
    dht = zero if x["dht"] is None else x["dht"].to(f64)
    o, ht, dq, dk, dv, dh0 = torch.zeros_like(v), zero.clone(), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), zero.clone()
    for n, (b, lo, hi) in enumerate(spans):
        S = h0[n].clone()
        for t in range(lo, hi):
            S = decay * S + k[b, t, :, :, None] * v[b, t, :, None, :]
            o[b, t] = x["scale"] * (S * q[b, t, :, :, None]).sum(-2)
            if backward:
                dq[b, t] = x["scale"] * (S * do[b, t, :, None, :]).sum(-1)
        ht[n] = S
        if backward:
            D = dht[n].clone()
            for t in reversed(range(lo, hi)):
                D = D + x["scale"] * q[b, t, :, :, None] * do[b, t, :, None, :]
                dk[b, t] = (D * v[b, t, :, None, :]).sum(-1)
                dv[b, t] = (D * k[b, t, :, :, None]).sum(-2)
                D = decay * D
            dh0[n] = D
    Hq = Hv // G
    return dict(o=o, ht=ht, dq=dq.unflatten(2, (Hq, G)).sum(3), dk=dk.unflatten(2, (Hq, G)).sum(3), dv=dv, dh0=dh0)


def verify(name, got, ref, io):
    assert got.dtype == (f32 if name in ("ht", "dh0") else io)
    check(name, got, ref, io, got.dtype, tol=FP32_TOL if got.dtype == f32 else BF16_TOL)


CASES = [  # B, T, Hq, Hv, K, V, dtype
    (1, 1, 1, 1, 64, 64, f32), (2, 65, 2, 4, 128, 128, f32), (1, 300, 1, 3, 64, 128, f32), (2, 33, 2, 2, 128, 64, f32),
    (1, 1, 1, 1, 128, 128, bf16), (2, 64, 2, 4, 128, 128, bf16), (3, 63, 1, 2, 128, 128, bf16), (1, 129, 2, 6, 128, 128, bf16),
    (2, 200, 2, 2, 64, 64, bf16), (1, 777, 2, 4, 64, 128, bf16), (2, 130, 1, 4, 128, 64, bf16), (40, 70, 2, 8, 128, 128, bf16),
]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case, packed):
    x = make(*case, seed=sum(case[:6]), packed=packed)
    o, ht = gdn.chunk_linear_attention(x["q"], x["k"], x["v"], x["g"], initial_state=x["h0"], output_final_state=True)
    ref = reference(x)
    verify("o", o, ref["o"], case[6])
    verify("ht", ht, ref["ht"], case[6])


@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case):
    x = make(*case, seed=1 + sum(case[:6]))
    leaves = [x[n].requires_grad_() for n in ("q", "k", "v", "h0")]
    o, ht = gdn.chunk_linear_attention(x["q"], x["k"], x["v"], x["g"], initial_state=x["h0"], output_final_state=True)
    grads = torch.autograd.grad([o, ht], leaves, [x["do"], x["dht"]])
    with torch.no_grad():
        ref = reference(x, backward=True)
    for name, got in zip(("dq", "dk", "dv", "dh0"), grads):
        verify(name, got, ref[name], case[6])


@pytest.mark.parametrize("G", [2, 3, 4, 5, 8])
@pytest.mark.parametrize("K", [64, 128])
def test_shared_heads(G, K):
    """Gradients of q and k are sums over the value heads that share them, in groups that the kernel sums itself and others."""
    x = make(2, 150, 2, 2 * G, K, 128, bf16, seed=G + K)
    leaves = [x[n].requires_grad_() for n in ("q", "k", "v", "h0")]
    o, ht = gdn.chunk_linear_attention(x["q"], x["k"], x["v"], x["g"], initial_state=x["h0"], output_final_state=True)
    grads = torch.autograd.grad([o, ht], leaves, [x["do"], x["dht"]])
    with torch.no_grad():
        ref = reference(x, backward=True)
    for name, got in zip(("dq", "dk", "dv", "dh0"), grads):
        verify(name, got, ref[name], bf16)


def packed_case(lengths, Hq, Hv, K, V, dtype, seed, T=None):
    ends = [0]
    for n in lengths:
        ends.append(ends[-1] + n)
    x = make(1, T or ends[-1], Hq, Hv, K, V, dtype, seed=seed, h0=False)
    gen = torch.Generator().manual_seed(seed + 1)
    x["h0"], x["dht"] = (torch.randn(len(lengths), Hv, K, V, generator=gen).cuda() for _ in range(2))
    return x, torch.tensor(ends, dtype=torch.int32).cuda(), [(0, a, b) for a, b in zip(ends, ends[1:])]


PACKED = [  # lengths, Hq, Hv, K, V, dtype
    ([5, 0, 1, 130, 64], 2, 4, 128, 128, bf16), ([300], 1, 2, 128, 128, bf16), ([64, 65, 63], 2, 2, 64, 128, bf16),
    ([1500, 10, 3, 200, 0, 70, 1], 4, 8, 128, 128, bf16), ([40, 90], 1, 3, 64, 64, f32), ([900, 0, 31, 700, 2], 2, 4, 128, 64, f32),
    ([3, 1] * 30 + [100], 1, 2, 128, 128, bf16), ([2100, 40, 40, 300], 24, 24, 64, 64, bf16),
]


@pytest.mark.parametrize("case", PACKED, ids=lambda c: "%d_%s" % (len(c[0]), "_".join(map(str, c[1:]))))
def test_packed(case):
    x, cu, spans = packed_case(*case, seed=len(case[0]))
    leaves = [x[n].requires_grad_() for n in ("q", "k", "v", "h0")]
    o, ht = gdn.chunk_linear_attention(x["q"], x["k"], x["v"], x["g"], initial_state=x["h0"], output_final_state=True, cu_seqlens=cu)
    grads = torch.autograd.grad([o, ht], leaves, [x["do"], x["dht"]])
    with torch.no_grad():
        ref = reference(x, spans, backward=True)
    verify("o", o, ref["o"], case[5])
    verify("ht", ht, ref["ht"], case[5])
    for name, got in zip(("dq", "dk", "dv", "dh0"), grads):
        verify(name, got, ref[name], case[5])


def call(x, **kw):
    return gdn.chunk_linear_attention(x["q"], x["k"], x["v"], x["g"], initial_state=x["h0"], output_final_state=True, **kw)


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_no_decay_scale_and_no_final_state(dtype):
    x = make(2, 200, 2, 4, 128, 64, dtype, seed=5)
    x["g"], x["scale"] = None, 0.25
    o, none = gdn.chunk_linear_attention(x["q"], x["k"], x["v"], scale=0.25)
    assert none is None
    x["h0"] = None
    verify("o", o, reference(x)["o"], dtype)
    x["g"] = torch.zeros(4, device="cuda", dtype=torch.float64)
    assert torch.equal(gdn.chunk_linear_attention(x["q"], x["k"], x["v"], x["g"], scale=0.25)[0], o)


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_decays_at_their_ends(dtype):
    """A head that keeps nothing, heads that keep almost nothing and almost everything, over many chunks."""
    x = make(1, 1000, 4, 4, 128, 128, dtype, seed=6)
    x["g"] = torch.tensor([-float("inf"), -60.0, -1e-6, 0.0], device="cuda")
    leaves = [x[n].requires_grad_() for n in ("q", "k", "v", "h0")]
    o, ht = call(x)
    grads = torch.autograd.grad([o, ht], leaves, [x["do"], x["dht"]])
    with torch.no_grad():
        ref = reference(x, backward=True)
    for name, got in zip(("o", "ht", "dq", "dk", "dv", "dh0"), (o, ht) + grads):
        for h in range(4):  # heads differ by orders of magnitude: each by itself
            if name in ("ht", "dh0"):
                verify(name, got[:, h], ref[name][:, h], dtype)
                continue
            # Where nothing is kept, dht reaches the last token alone: its dv is a sum of 128 products of numbers of size 1,
            # RMS sqrt(128) = 11.3, of which fp32 sums may lose 128 * 2^-24 * (128 * 0.64) = 6e-4 at worst, while the other
            # tokens' RMS is 1: the last token by itself too.
            verify(name, got[:, :-1, h], ref[name][:, :-1, h], dtype)
            verify(name, got[:, -1:, h], ref[name][:, -1:, h], dtype)


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_layouts(dtype):
    """Heads before tokens, rows off 16-byte boundaries, widths reversed, inputs shared by the batch, an offset state."""
    x = make(2, 150, 2, 4, 64, 128, dtype, seed=7)
    x["k"] = x["k"][:1].expand(2, -1, -1, -1)
    ref = reference(x, backward=True)
    q = x["q"].transpose(1, 2).contiguous().transpose(1, 2)
    v = torch.zeros(2, 150, 4, 131, dtype=dtype, device="cuda")[..., 3:]
    v.copy_(x["v"])
    flat = torch.empty(x["h0"].numel() + 1, device="cuda")[1:]
    h0 = flat.view_as(x["h0"]).copy_(x["h0"])
    do = x["do"].transpose(-1, -2).contiguous().transpose(-1, -2)
    o, ht = gdn.chunk_linear_attention_fwd(q, x["k"], v, x["g"], initial_state=h0)
    verify("o", o, ref["o"], dtype)
    verify("ht", ht, ref["ht"], dtype)
    grads = gdn.chunk_linear_attention_bwd(q, x["k"], v, x["g"], do, x["dht"], initial_state=h0)
    for name, got in zip(("dq", "dk", "dv", "dh0"), grads):
        verify(name, got, ref[name], dtype)


def test_gradient_of_a_sum():
    """The gradient of a sum comes expanded, all strides 0; and only some inputs may ask for theirs."""
    x = make(1, 90, 1, 2, 128, 128, bf16, seed=8)
    x["do"] = torch.ones_like(x["do"])
    with torch.no_grad():
        ref = reference(dict(x, dht=None), backward=True)
    x["k"].requires_grad_()
    call(x)[0].sum().backward()
    verify("dk", x["k"].grad, ref["dk"], bf16)
    x["h0"].requires_grad_()
    (dh0,) = torch.autograd.grad(call(x)[0].sum(), x["h0"])
    verify("dh0", dh0, ref["dh0"], bf16)
    x["do"] = torch.zeros_like(x["do"])
    with torch.no_grad():
        ref = reference(x, backward=True)
    dk, dh0 = torch.autograd.grad(call(x)[1], (x["k"], x["h0"]), x["dht"])
    verify("dk", dk, ref["dk"], bf16)
    verify("dh0", dh0, ref["dh0"], bf16)


def test_differences():
    """Gradients against differences of the call itself, in fp32: the function is linear in each input alone, so that a
    difference has no error of its own but the outputs' roundings (2^-24 of sums of a few thousand terms of size 1)."""
    x = make(1, 70, 1, 2, 64, 64, f32, seed=9)
    leaves = [x[n].requires_grad_() for n in ("q", "k", "v", "h0")]
    grads = torch.autograd.grad(list(call(x)), leaves, [x["do"], x["dht"]])
    gen = torch.Generator().manual_seed(1)
    with torch.no_grad():
        def value():
            o, ht = call(x)
            return float((o.double() * x["do"]).sum() + (ht.double() * x["dht"]).sum())

        for name, grad in zip(("q", "k", "v", "h0"), grads):
            step = torch.randn(x[name].shape, generator=gen).cuda()
            here = x[name].detach().clone()
            x[name].copy_(here + step)
            up = value()
            x[name].copy_(here - step)
            down = value()
            x[name].copy_(here)
            want = float((grad.double() * step).sum())
            size = float(grad.double().norm() * step.double().norm())
            assert abs((up - down) / 2 - want) <= 1e-5 * size


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_nothing_to_do(dtype):
    x = make(2, 0, 1, 2, 64, 128, dtype, seed=10)
    leaves = [x[n].requires_grad_() for n in ("q", "k", "v", "h0")]
    o, ht = call(x)
    assert o.shape == (2, 0, 2, 128) and torch.equal(ht, x["h0"])
    grads = torch.autograd.grad([o, ht], leaves, [x["do"], x["dht"]])
    assert grads[0].shape == x["q"].shape and torch.equal(grads[3], x["dht"])
    x = make(0, 5, 1, 2, 64, 128, dtype, seed=10)
    o, ht = call(x)
    assert o.shape == (0, 5, 2, 128) and ht.shape == (0, 2, 64, 128)
    x = make(1, 9, 1, 2, 64, 128, dtype, seed=10, h0=False)
    o, ht = call(x, cu_seqlens=torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert (o == 0).all() and ht.shape[0] == 0


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_rows_outside_every_sequence(dtype):
    """Offsets that begin late, end early, fall or leave the tokens: such sequences are empty, unclaimed rows are 0."""
    T = 400
    x = make(1, T, 2, 4, 128, 128, dtype, seed=11, h0=False)
    cu = torch.tensor([7, 100, 90, 250, T + 5, T + 5, 300, 390], device="cuda")
    spans = [(0, 7, 100), (0, 0, 0), (0, 90, 250), (0, 0, 0), (0, 0, 0), (0, 0, 0), (0, 300, 390)]
    gen = torch.Generator().manual_seed(2)
    x["h0"], x["dht"] = (torch.randn(7, 4, 128, 128, generator=gen).cuda() for _ in range(2))
    spans[0] = (0, 7, 90)  # tokens 90 .. 99 are claimed twice: what they get is one or the other
    got = call(x, cu_seqlens=cu)[0]
    ref = reference(x, spans)["o"]
    sure = torch.ones(T, dtype=torch.bool)
    sure[90:100] = False
    check("o", got[:, sure], ref[:, sure], dtype, dtype, tol=FP32_TOL if dtype == f32 else BF16_TOL)
    assert (got[0, :7] == 0).all() and (got[0, 250:300] == 0).all() and (got[0, 390:] == 0).all()
    dq, dk, dv, dh0 = gdn.chunk_linear_attention_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], x["dht"], initial_state=x["h0"], cu_seqlens=cu)
    for d in (dq, dk, dv):
        assert (d[0, :7] == 0).all() and (d[0, 250:300] == 0).all() and (d[0, 390:] == 0).all() and d.isfinite().all()
    for n in (1, 3, 4, 5):
        assert torch.equal(dh0[n], x["dht"][n])


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_what_is_not_finite_stays_in_its_sequence(dtype):
    x, cu, spans = packed_case([70, 130, 61], 1, 2, 128, 128, dtype, seed=12)
    clean = call(x, cu_seqlens=cu)[0].clone()
    for name in ("q", "k", "v"):
        x[name][0, 70:200] = float("nan")
        x[name][0, 75] = float("inf")
    o, ht = call(x, cu_seqlens=cu)
    assert torch.equal(o[0, :70], clean[0, :70]) and torch.equal(o[0, 200:], clean[0, 200:])
    assert ht[1].isnan().any() and ht[0].isfinite().all() and ht[2].isfinite().all()
    b = make(2, 100, 1, 2, 128, 128, dtype, seed=13)
    clean = call(b)[0].clone()
    b["v"][1] = float("nan")
    o = call(b)[0]
    assert torch.equal(o[0], clean[0]) and o[1].isnan().any()
    b["v"][1] = 0
    b["v"][0, 64, 0] = float("nan")  # the second chunk: the first does not see it
    assert call(b)[0][0, :64].isfinite().all()


def test_streams_graphs_and_two_at_once():
    x, y = make(1, 1500, 2, 4, 128, 128, bf16, seed=14), make(3, 100, 2, 4, 128, 128, bf16, seed=15)
    want = [t.clone() for z in (x, y) for t in call(z)]
    back = [t.clone() for t in gdn.chunk_linear_attention_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], x["dht"], initial_state=x["h0"])]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(5):
        got = []
        for z, side in zip((x, y), sides):
            with torch.cuda.stream(side):
                got += call(z)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, ht = call(x)
        grads = gdn.chunk_linear_attention_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], x["dht"], initial_state=x["h0"])
    other = torch.cuda.CUDAGraph()
    with torch.cuda.graph(other):
        o2, ht2 = call(y)
    for _ in range(3):
        graph.replay()
        other.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(ht, want[1]) and torch.equal(o2, want[2]) and torch.equal(ht2, want[3])
    assert all(torch.equal(a, b) for a, b in zip(grads, back))


def test_rows_beyond_32_bit_offsets():
    """v and o of more than 2^31 values: the last rows are those of the same sequence by itself."""
    B, T, Hv = 2, 70000, 128
    gen = torch.Generator(device="cuda").manual_seed(16)
    v = torch.randn(B, T, Hv, 128, device="cuda", generator=gen, dtype=bf16)
    assert v.numel() > 2 ** 31
    q, k = (torch.randn(B, T, 1, 128, device="cuda", generator=gen, dtype=bf16) for _ in range(2))
    g = torch.full((Hv,), -0.1, device="cuda")
    o, ht = gdn.chunk_linear_attention(q, k, v, g, output_final_state=True)
    tail = 640  # e^-64 of what came before is left: nothing
    o2, ht2 = gdn.chunk_linear_attention(q[1:, -tail:], k[1:, -tail:], v[1:, -tail:], g, output_final_state=True)
    a, b = o[1, -64:].float(), o2[0, -64:].float()
    assert (a - b).abs().max() <= 2 * 2 ** -8 * b.abs().max()
    check("ht", ht[1], ht2[0], f32, f32, tol=FP32_TOL)


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_continues(dtype):
    """A prompt in two parts, then token by token: the same as the whole, and the same states."""
    x = make(2, 203, 2, 4, 128, 128, dtype, seed=17)
    ref = reference(x)
    part = {n: x[n][:, :130] for n in ("q", "k", "v")}
    o1, s = call(dict(x, **part))
    part = {n: x[n][:, 130:200] for n in ("q", "k", "v")}
    o2, s = call(dict(x, h0=s, **part))
    rest = [x[n][:, 200:] for n in ("q", "k", "v")]
    o3 = gdn.recurrent_linear_attention(*rest, x["g"], s)
    verify("o", torch.cat([o1, o2, o3], 1), ref["o"], dtype)
    verify("ht", s, ref["ht"], dtype)


def test_misaligned_rows_in_c():
    """bf16 that the tensor cores' kernel does not take: the CUDA cores' one takes it (Python copies it instead)."""
    import ctypes as C
    lib = gdn.load_library()
    B, T, Hq, Hv, K, V = 1, 100, 1, 2, 64, 128
    x = make(B, T, Hq, Hv, K, V, bf16, seed=18)

    class S(C.Structure):
        _fields_ = [(n, C.c_int64) for n in ("batch", "token", "head")]

    class P(C.Structure):
        _fields_ = ([(n, C.c_int64) for n in ("B", "T", "Hq", "Hv", "K", "V", "n_seqs")] + [("cu", C.c_void_p), ("io", C.c_int), ("scale", C.c_float)] +
                    [(n, S) for n in ("q", "k", "v", "d_o")])

    side = torch.zeros(B, T, 2 * Hq * K + Hv * V + 3, dtype=bf16, device="cuda")
    q, k = side[..., 1:1 + K].view(B, T, 1, K), side[..., 1 + K:1 + 2 * K].view(B, T, 1, K)
    v = side[..., 1 + 2 * K:1 + 2 * K + Hv * V].unflatten(2, (Hv, V))
    for name, y in (("q", q), ("k", k), ("v", v)):
        y.copy_(x[name])
    p = P(B, T, Hq, Hv, K, V, B, None, 1, x["scale"], *(S(*y.stride()[:3]) for y in (q, k, v)), S(*x["do"].stride()[:3]))
    lib.gdn_linear_bwd_workspace_bytes.restype = C.c_size_t
    ws = torch.empty(lib.gdn_linear_bwd_workspace_bytes(C.byref(p)), dtype=torch.uint8, device="cuda")
    o, ht = torch.empty_like(x["v"]), torch.empty_like(x["h0"])
    out = [torch.empty_like(x[n]) for n in ("q", "k", "v", "h0")]
    at = lambda t: C.c_void_p(t.data_ptr())  # noqa: E731
    stream = C.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert lib.gdn_linear_fwd(C.byref(p), at(q), at(k), at(v), at(x["g"]), at(x["h0"]), at(o), at(ht), at(ws), C.c_size_t(ws.numel()), stream) == 0
    assert lib.gdn_linear_bwd(C.byref(p), at(q), at(k), at(v), at(x["g"]), at(x["h0"]), at(x["do"]), at(x["dht"]), *map(at, out), at(ws),
                              C.c_size_t(ws.numel()), stream) == 0
    ref = reference(x, backward=True)
    for name, got in zip(("o", "ht", "dq", "dk", "dv", "dh0"), [o, ht] + out):
        verify(name, got, ref[name], bf16)


@pytest.mark.parametrize("case", [(2, 1000, 4, 8, 64, 64), (1, 200, 4, 8, 128, 128), (1, 193, 2, 4, 128, 64), (1, 260, 1, 2, 64, 128)], ids=str)
def test_fp32_in_segments(case):
    x = make(*case, f32, seed=19)
    leaves = [x[n].requires_grad_() for n in ("q", "k", "v", "h0")]
    o, ht = call(x)
    grads = torch.autograd.grad([o, ht], leaves, [x["do"], x["dht"]])
    with torch.no_grad():
        ref = reference(x, backward=True)
    for name, got in zip(("o", "ht", "dq", "dk", "dv", "dh0"), (o, ht) + grads):
        verify(name, got, ref[name], f32)


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_sequences_that_are_one(dtype):
    """Offsets that name the same tokens twice, of sequences that would each be cut: more segments than there can be."""
    T = 6000
    x = make(1, T, 2, 32 if dtype == bf16 else 8, 64, 64, dtype, seed=20, h0=False)
    cu = torch.tensor([0, T, 0, T, 0], device="cuda")
    o, ht = gdn.chunk_linear_attention(x["q"], x["k"], x["v"], x["g"], output_final_state=True, cu_seqlens=cu)
    one, state = gdn.chunk_linear_attention(x["q"], x["k"], x["v"], x["g"], output_final_state=True)
    # two answers, each off by its tolerance and its rounding
    tol, half = (FP32_TOL, 2.0 ** -24) if dtype == f32 else (BF16_TOL, 2.0 ** -8)
    a, b = o.double(), one.double()
    assert ((a - b).abs() <= 2 * (tol * b.square().mean().sqrt() + half * torch.maximum(a.abs(), b.abs()))).all()
    for n in (0, 2):
        check("ht", ht[n], state[0], f32, f32, tol=2 * FP32_TOL)
    assert (ht[1] == 0).all() and (ht[3] == 0).all()
