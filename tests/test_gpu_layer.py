"""The convolution, the scan and the verification as a serving loop uses them:
after one another and in front of the delta rule, over drafted tokens, captured
into graphs, on other streams and from several threads."""
import threading

import numpy as np
import pytest
import torch

import _layer_ref as R
import linear_attention_recurrent_gb300 as lar

pytestmark = pytest.mark.gpu


def test_conv_feeds_the_delta_rule(cuda_device):
    """Packed q, k, v through the convolution, its output's slices into gdn_prefill
    and gdn_decode: a prompt and two tokens in those calls equal the whole in one."""
    dev, H, HV, K, L = cuda_device, 1, 2, 128, 45
    g = torch.Generator().manual_seed(1)
    C = 2 * H * K + HV * K
    x = torch.randn(L, C, generator=g).to(dev)
    w, b = (0.5 * torch.randn(C, 4, generator=g)).to(dev), torch.randn(C, generator=g).to(dev)
    gate, beta = -torch.rand(L, HV, generator=g).to(dev), torch.rand(L, HV, generator=g).to(dev)
    cpool, spool = torch.zeros(3, 3, C, device=dev), torch.zeros(3, HV, K, K, device=dev)
    idx = lambda i: torch.tensor([i], device=dev)  # noqa: E731

    def heads(y):
        return (y[..., :H * K].unflatten(-1, (H, K)), y[..., H * K:2 * H * K].unflatten(-1, (H, K)),
                y[..., 2 * H * K:].unflatten(-1, (HV, K)))

    def prompt(lo, hi, src, dst):
        off = torch.tensor([0, hi - lo], device=dev)
        y = lar.conv_prefill(x[lo:hi], w, cpool, off, idx(src), idx(dst), bias=b, silu=True)
        return lar.gdn_prefill(*heads(y), gate[lo:hi], beta[lo:hi], spool, off, idx(src), idx(dst), qk_l2norm=True)

    whole = prompt(0, L, -1, 0)
    part = [prompt(0, L - 2, -1, 1)]
    for t in (L - 2, L - 1):
        y = lar.conv_decode(x[t:t + 1], w, cpool, idx(1), bias=b, silu=True)
        part.append(lar.gdn_decode(*heads(y), gate[t:t + 1], beta[t:t + 1], spool, idx(1), qk_l2norm=True))
    assert torch.equal(cpool[0], cpool[1])
    # the chunked and the recurrent form differ by rounding, as their own tests allow
    torch.testing.assert_close(torch.cat(part), whole, rtol=1e-4, atol=1e-5)
    torch.testing.assert_close(spool[1], spool[0], rtol=1e-4, atol=1e-5)


class Layer:
    """A convolution and a scan behind it, with their states in pools of the same slots."""

    def __init__(self, dev, D=96, N=16, slots=64, seed=0):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g).to(dev)  # noqa: E731
        self.D, self.N = D, N
        self.w, self.b = 0.5 * r(D, 4), r(D)
        self.A, self.skip, self.bias = -torch.exp(r(D, N)), r(D), r(D) - 2
        self.cpool, self.spool = torch.zeros(slots, 3, D, device=dev), torch.zeros(slots, D, N, device=dev)

    def __call__(self, f, kind, **where):
        """f: x, dt, z, B, C of the tokens."""
        u = getattr(lar, "conv_" + kind)(f["x"], self.w, self.cpool, bias=self.b, silu=True, **where)
        return getattr(lar, "ssm_" + kind)(u, f["dt"], self.A, f["B"], f["C"], self.spool, D=self.skip, z=f["z"],
                                           dt_bias=self.bias, dt_softplus=True, **where)

    def reference(self, f, T):
        c = {k: R.f64(v) for k, v in f.items()}
        u, e, _ = R.conv_tokens(c["x"][:T], R.f64(self.w), R.f64(self.b), np.zeros((3, self.D)), True)
        out, _, hs, _ = R.ssm_tokens(u, c["dt"][:T], R.f64(self.A), c["B"][:T], c["C"][:T], np.zeros((self.D, self.N)),
                                     D=R.f64(self.skip), z=c["z"][:T], dt_bias=R.f64(self.bias), soft=True)
        return out, hs


def features(dev, lead, D, N, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g).to(dev)  # noqa: E731
    return dict(x=r(*lead, D), dt=r(*lead, D), z=r(*lead, D), B=r(*lead, 1, N), C=r(*lead, 1, N))


def test_drafted_steps(cuda_device):
    """A prompt, then steps of drafted tokens: each step runs all of its tokens into
    per-token slots, spec_verify says how many stand, and the next step starts from
    the state of the last of those.  What stands equals one pass over exactly the
    tokens that were kept."""
    dev, B, T, V, L0, steps = cuda_device, 4, 4, 50, 9, 5
    layer = Layer(dev, slots=B * (T + 1) + 1)
    vocab = features(dev, (V,), layer.D, layer.N, 5)       # a token's features
    g = torch.Generator().manual_seed(6)
    rows = torch.arange(B * T, device=dev).view(B, T)
    seq = torch.randint(V, (B, L0), generator=g)
    at = lambda ids: {k: v[ids.to(dev)] for k, v in vocab.items()}  # noqa: E731
    # the prompt leaves its state where an accepted count of 1 finds it
    flat = at(seq.reshape(-1))
    layer(flat, "prefill", cu_seqlens=torch.arange(0, B * L0 + 1, L0, device=dev), read_idx=torch.full((B,), -1, device=dev),
          write_idx=rows[:, 0])
    kept = [s.tolist() for s in seq]
    outs = [[] for _ in range(B)]
    acc = torch.ones(B, dtype=torch.int32, device=dev)
    last = torch.randint(V, (B,), generator=g)
    for i in range(steps):
        draft = torch.randint(V, (B, T - 1), generator=g)
        ids = torch.cat([last[:, None], draft], 1)
        out = layer(at(ids), "decode_tokens", state_idx=rows, num_accepted=acc)
        p = torch.softmax(torch.randn(B, T, V, generator=g), -1)
        q = torch.softmax(torch.randn(B, T - 1, V, generator=g), -1)
        u, v = torch.rand(B, T - 1, generator=g), torch.rand(B, generator=g)
        acc, toks = lar.spec_verify(draft.to(dev), p.to(dev), u.to(dev), v.to(dev), draft_probs=q.to(dev))
        ra, rt = R.verify(draft.tolist(), R.f64(p), R.f64(u), R.f64(v), R.f64(q))
        assert np.array_equal(acc.cpu(), ra) and np.array_equal(toks.cpu(), rt)
        for b in range(B):
            n = int(acc[b])
            outs[b].append(out[b, :n])
            kept[b] += ids[b, :n].tolist()
        last = toks.cpu().gather(1, acc.cpu().long()[:, None] - 1)[:, 0].long()
    for b in range(B):
        ref, hs = layer.reference(at(torch.tensor(kept[b])), len(kept[b]))
        got = torch.cat(outs[b]).cpu().double().numpy()
        np.testing.assert_allclose(got, ref[L0:], rtol=1e-4, atol=1e-4)
        state = layer.spool[rows[b, int(acc[b]) - 1]]
        np.testing.assert_allclose(R.f64(state), hs[-1], rtol=1e-4, atol=1e-4)


def prepared(dev, layer, f, slots, stream, out):
    """A decode step of the layer as two prepared calls."""
    u = torch.empty_like(f["x"])
    a = lar.PreparedCall("conv", x=f["x"], weight=layer.w, bias=layer.b, pool=layer.cpool, out=u, silu=True,
                         stream=stream, read_idx=slots)
    b = lar.PreparedCall("ssm", x=u, dt=f["dt"], A=layer.A, B=f["B"], C=f["C"], D=layer.skip, z=f["z"],
                         dt_bias=layer.bias, pool=layer.spool, out=out, dt_softplus=True, stream=stream, read_idx=slots)
    return lambda: (a(), b())


def test_graphs_and_streams(cuda_device):
    """Steps captured into two graphs that replay in turn on two streams, against the
    same steps run eagerly: bit-identical."""
    dev, B = cuda_device, 3
    layers = [Layer(dev, seed=7), Layer(dev, seed=7)]
    f = [features(dev, (B, 1), 96, 16, 8 + i) for i in range(2)]
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    slots = [torch.arange(B, device=dev) + B * i for i in range(2)]
    res = []
    for mode, layer in zip(("graph", "eager"), layers):
        outs = [torch.empty_like(f[i]["x"]) for i in range(2)]
        calls = [prepared(dev, layer, f[i], slots[i], streams[i], outs[i]) for i in range(2)]
        torch.cuda.synchronize()
        for i in range(2):
            calls[i]()
        torch.cuda.synchronize()
        if mode == "graph":
            graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
            for i in range(2):
                with torch.cuda.graph(graphs[i], stream=streams[i]):
                    for _ in range(3):
                        calls[i]()
            for _ in range(4):
                for i in range(2):
                    with torch.cuda.stream(streams[i]):
                        graphs[i].replay()
        else:
            for i in range(2):
                for _ in range(12):
                    calls[i]()
        torch.cuda.synchronize()
        res.append((outs, layer.cpool, layer.spool))
    for a, b in zip(res[0][0], res[1][0]):
        assert torch.equal(a, b)
    assert torch.equal(res[0][1], res[1][1]) and torch.equal(res[0][2], res[1][2])


def test_captured_prefill_and_verify(cuda_device):
    """Prompts and the verification captured; replays see the new contents of the
    buffers, offsets and counts among them."""
    dev, D, N, tok = cuda_device, 200, 16, 700
    layer = Layer(dev, D=D, slots=6)
    st = torch.cuda.Stream(dev)
    f = features(dev, (tok,), D, N, 3)
    off = torch.tensor([0, 300, tok], device=dev)
    read, write = torch.tensor([-1, -1], device=dev), torch.tensor([0, 1], device=dev)
    u, out = torch.empty(tok, D, device=dev), torch.empty(tok, D, device=dev)
    p = torch.softmax(torch.randn(2, 3, 999, device=dev), -1)
    draft, ua, us = torch.zeros(2, 2, dtype=torch.int32, device=dev), torch.rand(2, 2, device=dev), torch.rand(2, device=dev)
    acc, toks = torch.empty(2, dtype=torch.int32, device=dev), torch.empty(2, 3, dtype=torch.int32, device=dev)
    where = dict(cu_seqlens=off, read_idx=read, write_idx=write, prefill=True, stream=st)
    calls = [lar.PreparedCall("conv", x=f["x"], weight=layer.w, bias=layer.b, pool=layer.cpool, out=u, silu=True, **where),
             lar.PreparedCall("ssm", x=u, dt=f["dt"], A=layer.A, B=f["B"], C=f["C"], D=layer.skip, z=f["z"],
                              dt_bias=layer.bias, pool=layer.spool, out=out, dt_softplus=True, **where),
             lar.PreparedCall("verify", draft_tokens=draft, target_probs=p, u_accept=ua, u_sample=us,
                              num_accepted=acc, tokens=toks, stream=st)]
    torch.cuda.synchronize()
    for c in calls:
        c()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        for c in calls:
            c()
    for k in range(2):
        off.copy_(torch.tensor([0, 1 + k, tok - 5 * k]))
        f["x"].normal_()
        ua.uniform_()
        us.uniform_()
        draft.random_(0, 999)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [out.clone(), layer.spool.clone(), acc.clone(), toks.clone()]
        out.zero_()
        ref = layer(f, "prefill", cu_seqlens=off, read_idx=read, write_idx=write)
        end = int(off[-1])
        a2, t2 = lar.spec_verify(draft, p, ua, us)
        assert torch.equal(got[0][:end], ref[:end]) and torch.equal(got[1], layer.spool)
        assert torch.equal(got[2], a2) and torch.equal(got[3], t2)


def test_several_threads(cuda_device):
    """Threads with streams and slots of their own, at once, against one after another."""
    dev, B, n = cuda_device, 2, 4
    layers = [Layer(dev, seed=2), Layer(dev, seed=2)]
    f = [features(dev, (B, 1), 96, 16, i) for i in range(n)]
    errors = []
    torch.cuda.synchronize()

    def work(layer, i, stream):
        try:
            call = prepared(dev, layer, f[i], torch.arange(B, device=dev) + B * i, stream, torch.empty_like(f[i]["x"]))
            stream.wait_stream(torch.cuda.default_stream(dev))
            for _ in range(10):
                call()
            stream.synchronize()
        except Exception as e:   # seen below
            errors.append(e)

    threads = [threading.Thread(target=work, args=(layers[0], i, torch.cuda.Stream(dev))) for i in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(n):
        work(layers[1], i, torch.cuda.Stream(dev))
    assert not errors, errors
    assert torch.equal(layers[0].cpool, layers[1].cpool) and torch.equal(layers[0].spool, layers[1].spool)


def test_repeatable(cuda_device):
    """No atomics or races decide anything: the same call twice gives the same bits."""
    dev, D, N, tok = cuda_device, 520, 16, 3000
    f = features(dev, (tok,), D, N, 3)
    off = torch.tensor([0, 2500, 2501, tok], device=dev)
    p = torch.softmax(torch.randn(7, 3, 50000, device=dev), -1)
    ua, us = torch.rand(7, 2, device=dev), torch.rand(7, device=dev)
    draft = p[:, :2].argmax(-1)
    res = []
    for _ in range(3):
        layer = Layer(dev, D=D, slots=6)
        out = layer(f, "prefill", cu_seqlens=off, read_idx=torch.full((3,), -1, device=dev), write_idx=torch.arange(3, device=dev))
        res.append((out, layer.spool, layer.cpool) + lar.spec_verify(draft, p, ua, us))
    for r in res[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, res[0]))


def test_stepgraph_takes_the_new_calls(cuda_device):
    dev = cuda_device
    st = torch.cuda.Stream(dev)
    x = torch.randn(4, 64, device=dev)
    pool, out = torch.zeros(4, 3, 64, device=dev), torch.empty(4, 64, device=dev)
    w, idx = torch.randn(64, 4, device=dev), torch.arange(4, device=dev)
    host_in, host_out = torch.randn(4, 64).pin_memory(), torch.empty(4, 64).pin_memory()
    torch.cuda.synchronize()
    call = lar.PreparedCall("conv", x=x, weight=w, pool=pool, read_idx=idx, out=out, stream=st)
    graph = lar.StepGraph(call, copies_in=[(x, host_in)], copies_out=[(host_out, out)], stream=st)
    before = pool.clone()
    host_in.normal_()
    graph.replay()
    st.synchronize()
    ref = lar.conv_decode(host_in.to(dev), w, before, idx)
    assert torch.equal(host_out, ref.cpu()) and torch.equal(before, pool)


def test_prepared_call_refusals(cuda_device):
    t = torch.zeros(1, 8, device=cuda_device)
    with pytest.raises(ValueError):
        lar.PreparedCall("conv", x=t, scale=2.0)
    with pytest.raises(ValueError):
        lar.PreparedCall("conv", x=t, cu_seqlens=t)             # packed without prefill=True
    with pytest.raises(ValueError):
        lar.PreparedCall("conv", x=t, z=t)                      # a name that the call does not take
    with pytest.raises(ValueError):
        lar.PreparedCall("verify", target_probs=t, silu=True)
    with pytest.raises(ValueError):
        lar.PreparedCall("gdn", q=t, silu=True)
    call = lar.PreparedCall("conv", x=t, weight=t, pool=t, read_idx=t, out=t)
    with pytest.raises(lar.LarError):
        call()
