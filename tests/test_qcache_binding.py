"""QCache's checks of where its tensors lie, on the CPU: tensors and the library are stand-ins, so nothing is launched."""
import pytest
import torch

from mla_block_diffusion_gb300 import dspark as D


class Stand:
    """What the binding asks of a tensor."""

    def __init__(self, *shape, dtype=torch.int32, device=0):
        self.shape, self.dtype, self.at = torch.Size(shape), dtype, device
        self.is_cuda, self.device = device >= 0, f"cuda:{device}"

    def get_device(self):
        return self.at

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def stride(self):
        return tuple(self.shape[i + 1:].numel() for i in range(len(self.shape)))

    def data_ptr(self):
        return 0x100000


class Library:
    """Counts the calls that reach the library."""
    calls = 0

    def dspark_qcache_workspace_bytes(self, *a):
        return 1024

    def __getattr__(self, name):
        def call(*a):
            self.calls += 1
            return 0
        return call


@pytest.fixture
def reach(monkeypatch):
    lib, current = Library(), [0]
    monkeypatch.setattr(D, "lib", lambda: lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0])
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0)
    return lib, current


def parts(device):
    u8, f32 = dict(dtype=torch.uint8, device=device), dict(dtype=torch.float32, device=device)
    return dict(codes=[Stand(8, 64, 80, **u8)], scales=[Stand(8, **f32)], page_table=Stand(3, 4, device=device),
                workspace=Stand(1024, **u8))


def cache(device=0, **kw):
    return D.QCache(64, 16, **(parts(device) | kw))


def args(device=0):
    i = lambda *s: Stand(*s, device=device)  # noqa: E731
    bf = lambda *s: Stand(*s, dtype=torch.bfloat16, device=device)  # noqa: E731
    plan = dict(length=i(3), want=i(3), ring=i(8), ring_state=i(2), length_out=i(3), ring_state_out=i(2), cu_new=i(4),
                slots=i(9), positions=i(9), seg_row=i(5))
    append = dict(entries=bf(1, 9, 80), slots=i(9), seg_row=i(5))
    attend = dict(layer=0, q=bf(5, 4, 80), cu_q=i(4), length=i(3), o=bf(5, 4, 64),
                  lse=Stand(5, 4, dtype=torch.float32, device=device))
    return {"plan": plan, "append": append, "attend": attend}


@pytest.mark.parametrize("device", [0, 2])
def test_one_device_throughout(reach, device):
    lib, current = reach
    current[0] = device
    c = cache(device)
    for n, (name, kw) in enumerate(args(device).items()):
        getattr(c, name)(**kw)
        assert lib.calls == n + 1
    assert c.check() == 0


@pytest.mark.parametrize("name", ["codes", "scales", "page_table", "workspace"])
@pytest.mark.parametrize("device", [1, -1])
def test_cache_parts_elsewhere(reach, name, device):
    with pytest.raises(ValueError):
        cache(**{name: parts(device)[name]})


@pytest.mark.parametrize("call,name", [(c, n) for c, kw in args().items() for n in kw if n != "layer"])
@pytest.mark.parametrize("device", [1, -1])
def test_arguments_elsewhere(reach, call, name, device):
    c = cache()
    with pytest.raises(ValueError):
        getattr(c, call)(**(args()[call] | {name: args(device)[call][name]}))
    assert reach[0].calls == 0


@pytest.mark.parametrize("call", ["plan", "append", "attend", "check"])
def test_another_current_device(reach, call):
    lib, current = reach
    c = cache()
    current[0] = 1
    with pytest.raises(ValueError):
        getattr(c, call)(**args().get(call, {}))
    assert lib.calls == 0
