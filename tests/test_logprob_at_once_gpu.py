"""The log-probability operators called from several threads at once, and whole
autograd steps of theirs captured into a graph and replayed."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ce():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import softmax_cross_entropy_pass_gb300 as ce
    return ce


def same(a, b):
    return len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


def inputs(seed, n=640, v=9001, H=64, V=1100):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randint(0, V, (n,), generator=g, device="cuda")
    t[::5] = -100
    return dict(x=(torch.randn(n, v, generator=g, device="cuda") * 2).bfloat16(), t=t,
                short=torch.randn(n, V, generator=g, device="cuda"), adv=torch.randn(n, generator=g, device="cuda"),
                ref=-torch.rand(n, generator=g, device="cuda"), off=torch.tensor([0, 100, 250, 400, 600], device="cuda"),
                h=torch.randn(n, H, generator=g, device="cuda").bfloat16(),
                w=(torch.randn(V, H, generator=g, device="cuda") * 0.1).bfloat16())


def direct(ce, d):
    out = []
    for x in (d["x"], d["short"]):
        logp, ent, stats = ce.ce_token_logprob(x, d["t"])
        out += [logp, ent, ce.ce_token_logprob_backward(x, d["t"], stats, d["adv"], grad_entropy=d["ref"], grad=torch.empty_like(x))]
        out += ce.ce_policy_fwd_bwd(x, d["t"], d["adv"], ref_logp=d["ref"], kl_coef=0.1, entropy_coef=0.01, grad=torch.empty_like(x))
        out += ce.ce_preference_fwd_bwd(x, d["t"], d["off"], grad=torch.empty_like(x))
    for n in (7, 100, len(d["t"])):      # the few-rows kernel, one CTA a tile, CTA pairs
        h, t, a = d["h"][:n], d["t"][:n], d["adv"][:n]
        logp, ent, stats = ce.flce_token_logprob(h, d["w"], t)
        out += [logp, ent, *ce.flce_token_logprob_backward(h, d["w"], t, stats, a, grad_entropy=a)[:2]]
    return [o.clone() for o in out]


def test_threads_at_once(ce):
    """Four threads, each with its own stream and inputs: what each computes alone."""
    data = [inputs(s) for s in range(4)]
    alone = [direct(ce, d) for d in data]
    torch.cuda.synchronize()
    start, failed = threading.Barrier(4), []

    def work(i):
        try:
            start.wait()
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(6):
                    got = direct(ce, data[i])
                    torch.cuda.current_stream().synchronize()
                    if not same(got, alone[i]):
                        failed.append(f"thread {i} differs")
        except BaseException as e:  # noqa: BLE001
            failed.append(repr(e))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not failed, failed


def step(ce, d, scale, inplace):
    """One training step's gradients; new leaves every time, so that no graph of theirs is left over."""
    out = []
    for k in ("x", "short"):
        a = d[k].detach().clone().requires_grad_()
        loss = ce.policy_loss(a * 1, d["t"], d["adv"], ref_logp=d["ref"], kl_coef=0.1, entropy_coef=0.01, grad_output=scale,
                              inplace=inplace)
        out += [loss.detach(), *torch.autograd.grad(loss * scale, a)]
        loss = ce.preference_loss(a * 1, d["t"], d["off"], inplace=inplace)
        out += [loss.detach(), *torch.autograd.grad(loss * scale, a)]
        logp, ent = ce.token_logprob(a * 1, d["t"], with_entropy=True, inplace=inplace)
        out += [logp.detach(), *torch.autograd.grad((logp * d["adv"] + 0.1 * ent).sum(), a)]
    h, w = d["h"].detach().requires_grad_(), d["w"].detach().requires_grad_()
    logp = ce.linear_token_logprob(h, w, d["t"])
    return out + [logp.detach(), *torch.autograd.grad((logp * d["adv"]).sum(), [h, w])]


@pytest.mark.parametrize("inplace", [False, True])
def test_captured_training_step(ce, inplace):
    d, scale = inputs(11), torch.full((), 8.0, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(ce, d, scale, inplace)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(ce, d, scale, inplace)
    for seed in (12, 13):
        for k, v in inputs(seed).items():
            d[k].copy_(v)
        scale.fill_(float(seed))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        assert same(got, [o.detach() for o in step(ce, d, scale, inplace)])
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, outs)


def test_captured_without_rows(ce):
    """No rows at all, captured: the losses are written all the same."""
    x, t, z = torch.empty(0, 50, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    w, off = torch.randn(30, 64, device="cuda").bfloat16(), torch.zeros(3, dtype=torch.int64, device="cuda")
    loss, ploss, gw = (torch.full(s, 9.0, device="cuda") for s in ((1,), (1,), (30, 64)))
    ws, pws = ce.workspace(0), torch.empty(4096, dtype=torch.uint8, device="cuda")

    def run():
        ce.ce_policy_fwd_bwd(x, t, z, loss=loss, ws=ws)
        ce.ce_preference_fwd_bwd(x, t, off, loss=ploss, ws=pws)
        ce.flce_token_logprob_backward(w[:0], w, t, torch.empty(0, 4, device="cuda"), z, grad_weight=gw)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for o in (loss, ploss, gw):
        o.fill_(9.0)
    graph.replay()
    torch.cuda.synchronize()
    assert loss.item() == 0 and ploss.item() == 0 and (gw == 0).all()
