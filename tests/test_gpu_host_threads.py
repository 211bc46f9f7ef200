"""Calls from several host threads at once, each on its own stream."""
import threading

import pytest
import torch

import gated_delta_rule_91_b200 as gdr

pytestmark = pytest.mark.gpu


def together(*work):
    """Runs the callables in threads of their own; raises what any of them raised."""
    wrong, start = [], threading.Barrier(len(work))

    def run(f):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                f()
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=run, args=(f,)) for f in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if wrong:
        raise wrong[0]


def test_layer_norm_gradients_of_two_widths():
    """Widths that share a kernel and differ in the shared memory that they need of it."""
    def work(D):
        g = torch.Generator().manual_seed(D)
        h, dy = (torch.randn(64, D, generator=g).cuda() for _ in range(2))
        w = torch.ones(D, device="cuda")
        want = [u.clone() for u in gdr.gdr_layernorm_bwd(h, w, dy)]
        torch.cuda.synchronize()

        dx, dw, db = (torch.empty_like(u) for u in (h, w, w))
        L = gdr.lib()
        ws = torch.empty(L.gdr_layernorm_bwd_workspace_bytes(D), dtype=torch.uint8, device="cuda")

        def run():
            args = (64, D, gdr.GDR_F32, h.data_ptr(), w.data_ptr(), 1e-5, dy.data_ptr(), None, dx.data_ptr(), dw.data_ptr(),
                    db.data_ptr(), ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
            for _ in range(10000):  # the entry itself: little of a call is outside it
                gdr.check(L.gdr_layernorm_bwd(*args))
            torch.cuda.current_stream().synchronize()
            assert all(torch.equal(a, b) for a, b in zip((dx, dw, db), want))
        return run

    together(work(33), work(127), work(3))


def test_scans_of_several_sizes():
    from test_gpu_ssm import bwd, fwd, inputs

    def work(size):
        d = inputs(*size, "bf16", seed=sum(size))
        want = fwd(d) + tuple(bwd(d).values())
        torch.cuda.synchronize()

        def run():
            for _ in range(20):
                got = fwd(d) + tuple(bwd(d).values())
            torch.cuda.current_stream().synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        return run

    together(work((1, 700, 2, 1, 64, 128)), work((2, 300, 4, 2, 128, 128)), work((1, 130, 3, 1, 64, 64)))


@pytest.mark.parametrize("name", ["gdr_ssm_fwd", "gdr_ssm_bwd", "gdr_fwd", "gdr2_fwd"])
def test_the_first_cuda_call_of_a_thread(name):
    """A thread that has called nothing of CUDA yet, as an autograd thread may be: buffers are all there."""
    import synth
    from test_gpu_ssm import inputs

    d = inputs(1, 140, 2, 1, 64, 64, "bf16", seed=4)
    x = {k: v.cuda() if torch.is_tensor(v) else v
         for k, v in (synth.gdr2_inputs if name == "gdr2_fwd" else synth.gdr_inputs)(1, 70, 2, 128, 128, "bf16", seed=5).items()}
    ins = (d["x"], d["delta"], d["A"], d["Bm"], d["Cm"], d["D"], d["bias"], d["S0"])
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    o, S = torch.empty_like(x["v"]), torch.empty(1, 2, 128, 128, device="cuda")
    y, S_T = torch.empty(1, 140, 2, 64, dtype=torch.bfloat16, device="cuda"), torch.empty_like(d["S0"])
    call = {"gdr_ssm_fwd": lambda: gdr.gdr_ssm_fwd(*ins, softplus=True, y=y, S_T=S_T, workspace=ws),
            "gdr_ssm_bwd": lambda: tuple(gdr.gdr_ssm_bwd(*ins, d["dy"], softplus=True, workspace=ws).values()),
            "gdr_fwd": lambda: gdr.gdr_fwd(*(x[k] for k in ("q", "k", "v", "log_alpha", "beta")), o=o, S_T=S, workspace=ws),
            "gdr2_fwd": lambda: gdr.gdr2_fwd(*(x[k] for k in ("q", "k", "v", "log_alpha", "b", "w")), o=o, S_T=S, workspace=ws)}[name]
    want = [u.clone() for u in call()]
    torch.cuda.synchronize()
    got, wrong = [], []

    def run():
        try:
            got.extend(call())
        except Exception as e:  # noqa: BLE001
            wrong.append(e)

    thread = threading.Thread(target=run)
    thread.start()
    thread.join()
    torch.cuda.synchronize()
    assert not wrong, wrong[0]
    assert all(torch.equal(a, b) for a, b in zip(got, want))
