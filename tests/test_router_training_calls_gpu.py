"""Router-training calls from two host threads, with the same expert several
times in a row, and against the formula that the host tests differentiate."""
import threading

import numpy as np
import pytest
import torch

from mixture_experts_layer_15_amd import binding as B
import test_router_training_abi as formula
from test_router_training_gpu import STEPS, Router, Step, dlogits64, make_mask

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.load_library()


def test_two_threads_on_two_streams_give_single_thread_bits():
    """Steps of different types and sizes at the same time, each thread with its own stream and buffers."""
    steps = [Step(STEPS["bf16"], make_mask(STEPS["bf16"].T, "random", 2)), Step(STEPS["f32"])]
    torch.cuda.synchronize()   # uploads done before other streams read them
    alone = []
    for s in steps:
        s.run()
        alone.append(s.outputs())
    for rep in range(3):
        streams = [torch.cuda.Stream() for _ in steps]
        errors = []
        start = threading.Barrier(len(steps))

        def work(i):
            try:
                start.wait()
                for _ in range(10):
                    steps[i].run(stream=streams[i])
                streams[i].synchronize()
            except Exception as e:  # reported below, in the main thread
                errors.append(e)

        threads = [threading.Thread(target=work, args=(i,)) for i in range(len(steps))]
        for t in threads:
            t.start()
        for t in threads:
            t.join(timeout=60)
        assert not any(t.is_alive() for t in threads), "a thread did not finish"
        assert not errors, errors
        for s, a in zip(steps, alone):
            got = s.outputs()
            assert all(torch.equal(got[n], a[n]) for n in a), rep


@pytest.mark.parametrize("T", [300, 33000])
@pytest.mark.parametrize("k", [4, 24])
def test_an_expert_named_often_gives_the_same_bits_every_time(T, k):
    """Several slots of a row add to one value: always in the same order."""
    r = Router(T, 128, 24, k, "bf16", "random")
    r.idx[::2] = 5
    r.idx[1::3] = torch.arange(k, dtype=torch.int32) // 3
    first = r.run()
    r.check(first)
    for _ in range(8):
        got = r.run()
        assert all(torch.equal(got[n], first[n]) for n in first)


def test_library_against_the_formula_of_the_host_tests():
    """test_gradient_formula_against_differences checks this formula; here the kernel is held to it."""
    r = Router(213, 128, 20, 3, "bf16", "random")
    got = r.run(("dlogits",))["dlogits"].double().numpy()
    n = lambda t: t.double().numpy()  # noqa: E731
    mask = r.mask.numpy() != 0
    ref = formula.dlogits64(n(r.L), r.idx.numpy(), n(r.w), n(r.g), n(r.counts), int(r.n), n(r.dl), mask)
    _, bound = dlogits64(r.L, r.idx, r.w, r.g, r.counts, int(r.n), r.dl, r.mask, 20, 3)
    assert np.all(np.abs(got - ref) <= bound.numpy() + 1e-37)
