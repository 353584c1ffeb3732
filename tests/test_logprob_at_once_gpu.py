"""The log-probability operators called from several threads at once."""
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
