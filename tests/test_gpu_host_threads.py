"""Host threads that call the layer function's operators at once, each on a stream of its own.

A launch's shared memory goes by its problem, while the limit that a launch is held to belongs
to the kernel in the whole process: every thread here keeps changing sizes, so that a limit
set for one call would sooner or later refuse another's launch."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
ROUNDS = 200


@pytest.fixture(scope="module")
def mhc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from manifold_constrained_hyper_token_b200 import build
    build.build()
    import manifold_constrained_hyper_token_b200 as m
    return m


def _ffn(mhc, T, C, F, dtype):
    g = torch.Generator(device="cuda").manual_seed(T)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")
    args = [n(T, C), n(F, C) * C ** -0.5, n(F, C) * C ** -0.5, n(C, F) * F ** -0.5, n(T, C)]
    args = [a.to(dtype) for a in args]
    return lambda: (mhc.mhc_ffn(*args[:4]), *mhc.mhc_ffn_backward(*args))


def _norm(mhc, T, C, dtype):
    g = torch.Generator(device="cuda").manual_seed(C)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, gy, w, b = n(T, C).to(dtype), n(T, C).to(dtype), n(C), n(C)
    return lambda: (mhc.mhc_layer_norm(x, w, b), *mhc.mhc_layer_norm_backward(x, w, gy))


def _calls(mhc, which):
    if which == "ffn bf16":  # one CTA or two to an SM, rings of every depth
        return [_ffn(mhc, T, 264, 520, BF16) for T in (1, 40, 100, 129, 200, 256)]
    if which == "ffn f32":
        return [_ffn(mhc, T, 264, 520, F32) for T in (3, 9, 40, 70, 100, 128)]
    if which == "norm bf16":
        return [_norm(mhc, T, C, BF16) for T, C in ((40, 264), (40, 1032), (40, 8192), (40, 8200),
                                                    (40, 14336), (2401, 1032), (2401, 4096))]
    return [_norm(mhc, T, C, F32) for T, C in ((40, 264), (40, 512), (40, 1032), (40, 4096),
                                               (40, 4104), (40, 7168))]


@pytest.mark.parametrize("which", ["ffn bf16", "ffn f32", "norm bf16", "norm f32"])
def test_threads_that_change_sizes(mhc, which):
    calls = _calls(mhc, which)
    want = [c() for c in calls]
    torch.cuda.synchronize()
    found = []

    def work(k):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for r in range(ROUNDS):
                    i = (r * (k + 1) + k) % len(calls)
                    got = calls[i]()
                    if r % 20 == 0:
                        s.synchronize()
                        if not all(torch.equal(a, b) for a, b in zip(want[i], got)):
                            found.append(f"thread {k}: other bits from call {i}")
                            return
            s.synchronize()
        except Exception as e:
            found.append(f"thread {k}: {e}")

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not found, found
