"""GPU: what the binding of include/muonstep_train.h promises about buffers, streams and arguments."""

import gc
import threading
import weakref

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _small(n=40, v=300, d=64, seed=0):
    import torch
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, d, generator=g).bfloat16().cuda(), torch.randn(v, d, generator=g).bfloat16().cuda(),
            torch.randint(0, v, (n,), generator=g).cuda())


def test_one_shot_calls_share_no_workspace():
    """The buffers that muon_step's calls share, one for each stream, are not theirs."""
    import muon_optimizer_step_amd as ms
    from muon_optimizer_step_amd import api
    api._workspaces.clear()
    ms.linear_cross_entropy_grad(*_small(2000, 4000, 512))
    ms.linear_cross_entropy(*_small())
    assert not api._workspaces


def test_one_shot_calls_of_two_threads_on_one_stream():
    import torch
    import muon_optimizer_step_amd as ms
    inputs = [_small(600, 5000, 128, seed=1), _small(500, 7000, 136, seed=2)]
    want = [[x.clone() for x in ms.linear_cross_entropy_grad(*i)] for i in inputs]
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(2)

    def work(k):
        start.wait()
        kept = [ms.linear_cross_entropy_grad(*inputs[k]) for _ in range(50)]
        torch.cuda.synchronize()
        wrong.extend((k, n) for n, r in enumerate(kept) if not all(torch.equal(a, b) for a, b in zip(r, want[k])))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == []


def test_one_shot_call_in_a_graph_keeps_its_workspace():
    """Calls after the capture, larger ones on its stream and on many others, neither change what the graph computes nor
    lose memory to it."""
    import torch
    import muon_optimizer_step_amd as ms
    h, w, t = _small(300, 3000, 96)
    ms.linear_cross_entropy_grad(h, w, t)
    want = [x.clone() for x in ms.linear_cross_entropy_grad(h, w, t)]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        r = ms.linear_cross_entropy_grad(h, w, t)
    large = _small(4000, 9000, 256, seed=3)
    for s in [torch.cuda.Stream() for _ in range(6)] + [None]:
        if s is not None:
            s.wait_stream(torch.cuda.current_stream())
        ms.linear_cross_entropy_grad(*large, stream=s)
        torch.cuda.synchronize()
    others = [torch.full((1 << 20,), 7, dtype=torch.int32, device="cuda") for _ in range(64)]
    for k in range(4):
        for x in r:
            x.fill_(float("nan"))
        g.replay()
        float(torch.randn(1 << 16, device="cuda").sum())
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(r, want)), k
        assert all(bool((x == 7).all()) for x in others), k


def test_a_workspace_elsewhere_is_refused():
    import torch
    import muon_optimizer_step_amd as ms
    h, w, t = _small()
    need = 1 << 24
    for bad, error in ((torch.empty(need, dtype=torch.uint8), ValueError), (torch.empty(need, dtype=torch.uint8).pin_memory(), ValueError),
                       (torch.empty(4096, need // 2048, dtype=torch.uint8, device="cuda")[:, :need // 4096], ValueError),
                       (need, TypeError)):
        for call in (ms.linear_cross_entropy, ms.linear_cross_entropy_grad, ms.PreparedLinearCrossEntropy):
            with pytest.raises(error, match="workspace"):
                call(h, w, t, workspace=bad)
    a = ms.linear_cross_entropy(h, w, t, workspace=torch.empty(need // 4, device="cuda"))
    assert torch.equal(a.nll, ms.linear_cross_entropy(h, w, t).nll)


def test_prepared_adamw8_keeps_its_tensors():
    import torch
    import muon_optimizer_step_amd as ms
    x = lambda dtype=torch.float32: [torch.zeros(512, device="cuda", dtype=dtype)]  # noqa: E731
    params, grads, emas, copies = x(), x(), x(), x(torch.bfloat16)
    states = [ms.AdamW8State.zeros_like(params[0])]
    call = ms.PreparedAdamW8(params, grads, states, emas=emas, copies=copies)
    s = states[0]
    refs = [weakref.ref(t) for t in (params[0], grads[0], emas[0], copies[0], s.exp_avg, s.exp_avg_scale, s.rms, s.rms_scale)]
    for lst in (params, grads, states, emas, copies):
        lst.clear()
    s.exp_avg = s.exp_avg_scale = s.rms = s.rms_scale = None
    del s
    gc.collect()
    assert [i for i, r in enumerate(refs) if r() is None] == []
    call(lr=1e-3, step=1)


def test_a_single_row_has_no_row_stride():
    """The last token of one long sequence: a view whose stride is the sequence's."""
    import torch
    import muon_optimizer_step_amd as ms
    h, w, t = _small(1)
    wide = torch.as_strided(h, (1, 64), (1 << 23, 1))
    assert wide.stride(0) == 1 << 23
    a, b = ms.linear_cross_entropy(wide, w, t), ms.linear_cross_entropy(h, w, t)
    assert torch.equal(a.nll, b.nll) and torch.equal(a.lse, b.lse)


def test_scalars_of_numpy_and_torch():
    import torch
    import muon_optimizer_step_amd as ms
    rng = np.random.default_rng(0)
    p0, g = torch.from_numpy(rng.standard_normal(700)).float().cuda(), torch.from_numpy(rng.standard_normal(700)).float().cuda()
    out = []
    for f, i in ((float, int), (np.float64, np.int64), (torch.tensor, torch.tensor), (np.float32, np.int32)):
        p, s = p0.clone(), ms.AdamW8State.zeros_like(p0)
        ms.adamw8_step([p], [g], [s], lr=f(2.0 ** -7), betas=(f(0.5), f(0.75)), eps=f(2.0 ** -20), weight_decay=f(0.25),
                       step=i(3), seed=i(11), ema_decay=f(0.5))
        out.append((p, s.exp_avg.view(torch.uint8), s.rms.view(torch.uint8)))
    for o in out[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, out[0]))
    for step in ((1 << 32) + 3, 1 << 31):
        with pytest.raises(ValueError, match="32 bits"):
            ms.adamw8_step([p0], [g], [s], lr=0.0, step=step)


def test_inputs_dropped_after_a_call_on_another_stream():
    """The caller's references end before the stream gets to the call; what takes their memory's place must not show."""
    import torch
    import muon_optimizer_step_amd as ms
    h, w, t = _small(700, 3000, 128)
    weights = torch.rand(700, device="cuda") / 700
    want = [x.clone() for x in ms.linear_cross_entropy_grad(h, w, t, token_weights=weights)]
    p = torch.randn(50000, device="cuda")
    grad, m, v = torch.randn_like(p), torch.randn_like(p), torch.rand_like(p)
    state = ms.AdamW8State.from_moments(m, v)
    want_m, want_v = state.moments()
    p1 = p.clone()
    ms.adamw8_step([p1], [grad], [state], lr=0.1, step=3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def late(call, *tensors):
        """call(copies of the tensors) on the busy side stream; the copies' memory is taken over at once."""
        copies = [x.clone() for x in tensors]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(5_000_000)
        out = call(*copies)
        del copies
        junk = [torch.full_like(x, 0 if x.dtype == torch.int64 else float("nan")) for x in tensors for _ in range(3)]
        torch.cuda.synchronize()
        del junk
        return out

    r = late(lambda h, w, t, g: ms.linear_cross_entropy_grad(h, w, t, token_weights=g, stream=side), h, w, t, weights)
    assert all(torch.equal(a, b) for a, b in zip(r, want))
    s = late(lambda m, v: ms.AdamW8State.from_moments(m, v, stream=side), m, v)
    assert all(torch.equal(a, b) for a, b in zip(s.moments(), (want_m, want_v)))
    p2 = p.clone()
    late(lambda g: ms.adamw8_step([p2], [g], [s], lr=0.1, step=3, stream=side), grad)
    assert torch.equal(p1, p2)
