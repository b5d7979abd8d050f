"""The router by scores called as its documentation allows: buffers on 4 bytes, larger workspaces, two calls at once."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
B = pytest.importorskip("expert_cached_moe_amd.binding")
from test_gpu_route_scored import POISON, Router, cuda, draw  # noqa: E402

pytestmark = pytest.mark.gpu


def shifted(a, by):
    """The same numbers `by` elements behind a 16-byte boundary."""
    t = torch.zeros(a.size + by, device="cuda")
    t[by:] = cuda(a).reshape(-1)
    return t[by:]


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [3, 40, 2108])
@pytest.mark.parametrize("E,k,groups,keep", [(256, 8, 8, 4), (48, 6, 1, 1), (512, 16, 1, 1), (96, 3, 4, 2)])
def test_buffers_on_4_bytes(E, k, groups, keep, T, kind):
    logits, bias, dw = draw(T, E, T + E, True, k)
    r = Router(E, k, T, kind, groups, keep, 2, 1, 1.5)
    for a, b in ((1, 0), (0, 3), (2, 1)):
        for t in (r.ids, r.perm, r.inv):
            t.fill_(POISON)
        dl = shifted(logits, a)
        r.forward(dl, shifted(bias, b))
        ids = r.check(logits, bias)
        r.backward(dl, shifted(dw, b))
        r.check_gradient(logits, ids, dw)


@pytest.mark.parametrize("T", [5, 100, 2109])
def test_a_workspace_sized_for_more_tokens(T):
    E, k = 100, 5
    logits, bias, _ = draw(T, E, T)
    r = Router(E, k, T, "sigmoid", 4, 2, 2)
    for most in (T + 1, 1 << 15):
        r.ws = torch.full((B.moe_workspace_bytes(r.cfg, most),), 0xFF, dtype=torch.uint8, device="cuda")
        r.forward(cuda(logits), cuda(bias))
        r.check(logits, bias)


@pytest.mark.parametrize("T", [4, 300, 4100])
def test_two_calls_at_once(T):
    """Two streams, each with its own buffers and workspace."""
    E, k = 128, 8
    routers, inputs, streams = [], [], []
    for seed in (1, 2):
        logits, bias, dw = draw(T, E, seed, True, k)
        routers.append(Router(E, k, T, "sigmoid", 8, 4, 2, 1, 2.5))
        inputs.append((logits, bias, dw, cuda(logits), cuda(bias), cuda(dw)))
        streams.append(torch.cuda.Stream())
    torch.cuda.synchronize()
    for _ in range(10):
        for r, i, s in zip(routers, inputs, streams):
            r.forward(i[3], i[4], s)
            r.backward(i[3], i[5], s)
    torch.cuda.synchronize()
    for r, i in zip(routers, inputs):
        ids = r.check(i[0], i[1])
        r.check_gradient(i[0], ids, i[2])


def test_ids_of_a_token_that_are_all_outside():
    """No expert chosen: no gradient."""
    T, E, k = 7, 20, 3
    logits, _, dw = draw(T, E, 5, False, k)
    for kind in ("softmax", "sigmoid"):
        for renorm in (0, 1):
            r = Router(E, k, T, kind, renorm=renorm)
            r.ids[:T * k] = -1
            r.backward(cuda(logits), cuda(dw))
            torch.cuda.synchronize()
            assert np.array_equal(r.d[:T * E].cpu().numpy(), np.zeros(T * E, np.float32))
