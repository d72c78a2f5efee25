"""Host-side statuses and sizes of gbla_adamw_step and gbla_grad_norm (no GPU needed)."""
import ctypes

import pytest

from generative_retrieval_encoder_gb300 import build, gbla

FAKE, ODD = 1 << 20, (1 << 20) + 1  # addresses, never dereferenced
I, W, U, OK = gbla.GBLA_ERR_INVALID_ARG, gbla.GBLA_ERR_WORKSPACE, gbla.GBLA_ERR_UNSUPPORTED, gbla.GBLA_OK


@pytest.fixture(scope="module")
def L():
    build.build()
    return gbla.lib()


def tensors(count=2, **kw):
    t = (gbla.AdamWTensor * count)()
    for e in t:
        for k, v in {**dict(param=FAKE, grad=FAKE, m=FAKE, v=FAKE, n=100), **kw}.items():
            setattr(e, k, v)
    return t


def step(L, t, n=None, step=FAKE, norm=None, ws=FAKE, size=1 << 30, **cfg):
    c = gbla.AdamWConfig(**{**dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, max_norm=0.0, seed=0), **cfg})
    return L.gbla_adamw_step(t, len(t) if n is None else n, ctypes.byref(c), step, norm, ws, size, None)


def test_step_host_errors(L):
    for bad in (dict(param=None), dict(param=ODD), dict(grad=None), dict(grad=ODD), dict(m=None), dict(v=ODD), dict(param_dtype=2),
                dict(grad_dtype=-1), dict(n=-1), dict(n=1 << 41), dict(master=FAKE), dict(m_scale=FAKE), dict(v_scale=FAKE),
                dict(m_scale=ODD, v_scale=FAKE), dict(weight_decay=-1.0), dict(weight_decay=float("nan")),
                dict(param_dtype=1, master=ODD)):
        assert step(L, tensors(**bad)) == I, bad
    for bad in (dict(lr=-1.0), dict(lr=float("nan")), dict(lr=float("inf")), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(eps=0.0),
                dict(eps=float("nan")), dict(max_norm=-1.0), dict(max_norm=1.0), dict(max_norm=float("nan"), norm=FAKE), dict(step=None),
                dict(step=FAKE + 4), dict(norm=ODD), dict(n=-1)):
        assert step(L, tensors(), **bad) == I, bad
    assert L.gbla_adamw_step(None, 1, None, FAKE, None, FAKE, 1 << 30, None) == I
    assert L.gbla_adamw_step(tensors(), 2, None, FAKE, None, FAKE, 1 << 30, None) == I
    size = L.gbla_adamw_workspace_size(tensors(), 2)
    assert size > 0
    assert step(L, tensors(), ws=None) == W and step(L, tensors(), ws=FAKE + 16) == W and step(L, tensors(), size=64) == W
    assert step(L, tensors(300, n=1 << 40)) == U


def test_norm_host_errors_and_sizes(L):
    t = tensors(param=None, m=None, v=None)  # not read
    assert L.gbla_grad_norm(t, 2, None, FAKE, 1 << 30, None) == I
    assert L.gbla_grad_norm(t, 2, ODD, FAKE, 1 << 30, None) == I
    assert L.gbla_grad_norm(t, -2, FAKE, FAKE, 1 << 30, None) == I
    assert L.gbla_grad_norm(tensors(grad=ODD), 2, FAKE, FAKE, 1 << 30, None) == I
    assert L.gbla_grad_norm(t, 2, FAKE, None, 1 << 30, None) == W
    assert L.gbla_adamw_workspace_size(t, -1) == 0 and L.gbla_adamw_workspace_size(None, 3) == 0
    assert L.gbla_adamw_workspace_size(tensors(n=-1), 2) == 0
    big = tensors(400, n=1 << 20)
    assert L.gbla_adamw_workspace_size(big, 400) > L.gbla_adamw_workspace_size(t, 2) > 0
    assert L.gbla_adamw_workspace_size(None, 0) > 0


def test_binding_refuses_host_tensors(L):
    import torch
    p = [torch.zeros(4)]
    with pytest.raises(ValueError):
        gbla.gbla_adamw_plan(p, p, {"step": torch.zeros(1, dtype=torch.int64), "m": p, "v": p})
    with pytest.raises(ValueError):
        gbla.gbla_adamw_state(p, bits=16)


class Fake:
    """What the binding asks of a tensor, with an address that nothing reads."""
    is_cuda, made = True, 0

    def __init__(self, n, dtype):
        import torch
        Fake.made += 1
        self.n, self.dtype, self.device, self.shape, self.at = n, dtype, torch.device("cpu"), (n,), FAKE + (Fake.made << 16)

    def numel(self):
        return self.n

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.at


def fakes(sizes, dtype):
    return [Fake(n, dtype) for n in sizes]


def test_plan_keeps_its_tensors_alive(L):
    """Also where the caller puts others in the state's lists afterwards."""
    import gc
    import torch
    import weakref
    sizes, f32 = [100, 300], torch.float32
    P, G = fakes(sizes, torch.bfloat16), fakes(sizes, f32)
    st = {"step": Fake(1, torch.int64), "m": fakes(sizes, torch.float8_e4m3fn), "v": fakes(sizes, torch.float8_e4m3fn),
          "m_scale": fakes([1, 2], f32), "v_scale": fakes([1, 2], f32), "master": fakes(sizes, f32)}
    refs = [weakref.ref(t) for t in P + G + [st["step"]] + st["m"] + st["v"] + st["m_scale"] + st["v_scale"] + st["master"]]
    plan = gbla.gbla_adamw_plan(P, G, st)
    for k in ("m", "v", "m_scale", "v_scale", "master"):
        st[k][0] = None
    st.clear()
    P.clear()
    G.clear()
    gc.collect()
    assert all(r() is not None for r in refs)
    del plan
    gc.collect()
    assert not any(r() is not None for r in refs)


def test_gradients_by_name(L):
    """The name d<name> is a parameter's gradient unless another parameter has that name."""
    import torch
    f32 = torch.float32
    P = {"w": Fake(10, f32), "dw": Fake(10, f32), "lam": Fake(10, f32)}
    state = {"step": Fake(1, torch.int64), "m": fakes([10] * 3, f32), "v": fakes([10] * 3, f32)}
    G = {k: Fake(10, f32) for k in ("w", "dw", "dlam")}
    plan = gbla.gbla_adamw_plan(P, G, state)
    assert [t.grad for t in plan.tensors] == [G[k].at for k in ("w", "dw", "dlam")]
    for bad in ({k: G["w"] for k in ("dw", "ddw", "dlam")}, {k: G["w"] for k in ("w", "dw")}):
        with pytest.raises(ValueError, match="gradient of"):
            plan.set_grads(bad)
    assert [t.grad for t in plan.tensors] == [G[k].at for k in ("w", "dw", "dlam")]
