"""Host-side checks of the routed layer's entry points and of the AdamW step: struct layouts,
refusals (before any CUDA call), and the k range of the row exchange."""
import ctypes
import math

import pytest

P = ctypes.c_void_p(4096)      # aligned dummy addresses, never dereferenced
ODD = ctypes.c_void_p(4098)
FOUR = ctypes.c_void_p(4100)


@pytest.fixture(scope="module")
def moe():
    import sparse_mixture_experts_fwd_b200 as m
    return m


def rcfg(moe, **kw):
    base = dict(T=100, E=64, k=4)
    base.update(kw)
    return moe.make_route_config(base.pop("T"), base.pop("E"), base.pop("k"), **base)


def test_struct_sizes(moe):
    assert moe.lib.moe_route_config_size() == ctypes.sizeof(moe.RouteConfig) == 48
    assert moe.lib.moe_adamw_config_size() == ctypes.sizeof(moe.AdamWConfig) == 64


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -1), (dict(E=0), -1), (dict(E=257), -2), (dict(k=0), -2), (dict(k=17), -2),
    (dict(E=3, k=4), -1), (dict(num_groups=0, top_groups=1), -1), (dict(num_groups=7), -1),
    (dict(num_groups=64), -2), (dict(num_groups=8, top_groups=9), -1),
    (dict(num_groups=8, top_groups=0), -1), (dict(num_groups=32, group_top=3), -1),
    (dict(group_top=0), -1), (dict(E=32, num_groups=32, group_top=2), -1),
    (dict(k=9, num_groups=8, top_groups=1), -1), (dict(scale=math.inf), -1),
    (dict(scale=math.nan), -1), (dict(scale=1e300), -1), (dict(T=2 ** 29, k=4), -2),
])
def test_route_config_refusals(moe, kw, code):
    c = rcfg(moe, **kw)
    for call in (lambda: moe.lib.moe_route(ctypes.byref(c), P, P, P, P, None, None),
                 lambda: moe.lib.moe_route_backward(ctypes.byref(c), P, P, P,
                                                    ctypes.c_void_p(8192), None, None)):
        assert call() == code
        assert moe.lib.moe_last_error().decode() != ""


def test_route_enum_refusals(moe):
    for field, value in (("score", 2), ("renorm", 2), ("dtype", 5)):
        c = rcfg(moe)
        setattr(c, field, value)
        assert moe.lib.moe_route(ctypes.byref(c), P, P, P, P, None, None) == -1
    assert moe.lib.moe_route(None, P, P, P, P, None, None) == -1


def test_route_pointer_refusals(moe):
    c = rcfg(moe)
    r, b = moe.lib.moe_route, moe.lib.moe_route_backward
    ref = ctypes.byref(c)
    assert r(ref, None, P, P, P, None, None) == -1
    assert r(ref, P, P, None, P, None, None) == -1
    assert r(ref, P, P, P, None, None, None) == -1
    assert r(ref, FOUR, P, P, P, None, None) == -3
    assert r(ref, P, ODD, P, P, None, None) == -3
    assert r(ref, P, P, ODD, P, None, None) == -3
    assert b(ref, P, P, P, None, None, None) == -1
    assert b(ref, P, P, P, P, None, None) == -1        # dlogits is logits
    assert b(ref, P, P, P, FOUR, None, None) == -3
    assert b(ref, P, None, P, ctypes.c_void_p(8192), None, None) == -1
    empty = rcfg(moe, T=0)
    assert r(ctypes.byref(empty), None, None, None, None, None, None) == 0


def test_choice_range_of_the_row_exchange(moe):
    lib = moe.lib
    for k, code in ((0, -2), (17, -2), (16, -1), (3, -1)):
        c = moe.make_config(32, 64, 64, 32, k, 8)
        ref = ctypes.byref(c)
        # -1 for a valid k: the null argument is found after the config
        assert lib.moe_assign(ref, None, P, P, P, P, P, P, None, None) == code
        assert lib.moe_dispatch(ref, None, P, P, P, P, None, None) == code
        assert lib.moe_dispatch_backward(ref, None, P, P, P, P, None, None) == code
        assert lib.moe_combine(ref, None, P, P, P, P, P, None, None) == code
        assert lib.moe_combine_backward(ref, None, P, P, P, P, P, P, P, None, None) == code
        # everything else keeps one or two choices
        assert lib.moe_config_check(ref) == -2 and lib.moe_workspace_size(ref) == 0
    c = moe.make_config(32, 64, 128, 32, 8, 8)
    f = moe.ep_ffn_config(c, 1)
    assert (f.E, f.capacity, f.k, f.d_model, f.d_ff) == (32, 8, 1, 64, 128)
    moe.config_check(f)
    ref = ctypes.byref(c)
    assert lib.moe_combine_backward(ref, P, P, P, P, P, P, P, ODD, None, None) == -3
    assert lib.moe_combine_backward(ref, P, P, P, None, P, P, P, P, None, None) == -1
    assert lib.moe_dispatch_backward(ref, P, P, P, P, FOUR, None, None) == -3
    bad = moe.make_config(32, 64, 64, 2, 3, 8)         # k > E
    assert lib.moe_assign(ctypes.byref(bad), P, P, P, P, P, P, P, None, None) == -1


def arrays(n, value=4096, step=65536):
    a = (ctypes.c_void_p * n)(*[value + step * i for i in range(n)])
    return ctypes.cast(a, ctypes.c_void_p), a


def adamw_call(moe, n=2, check=False, lens=(100, 50), norm=None, step_lr=None, drop=(), **cfg):
    base = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, max_norm=1.0, step=1,
                grad_dtype=1, state_bits=32)
    base.update(cfg)
    c = moe.AdamWConfig(**base)
    le = (ctypes.c_int64 * max(1, len(lens)))(*lens)
    keep, args = [le], [ctypes.cast(le, ctypes.c_void_p)]
    for i, name in enumerate(("p", "g", "m", "v", "ms", "vs", "copy")):
        ptr, a = arrays(max(1, n), (1 << 24) * (i + 1))
        if name in drop:
            ptr = None
        keep.append(a)
        args.append(ptr)
    if check:
        return moe.lib.moe_adamw_check(ctypes.byref(c), n, *args), keep
    return moe.lib.moe_adamw_step(ctypes.byref(c), n, *args, norm, step_lr, None, None), keep


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), -1), (dict(n=4097, lens=(0,) * 4097), -2), (dict(lens=(-1, 5)), -1),
    (dict(beta1=1.0), -1), (dict(beta2=-0.1), -1), (dict(eps=0.0), -1), (dict(eps=1e-39), -1),
    (dict(eps=math.inf), -1), (dict(weight_decay=math.nan), -1), (dict(step=0), -1),
    (dict(lr=math.inf), -1), (dict(norm=P, max_norm=0.0), -1), (dict(norm=P, max_norm=math.inf), -1),
    (dict(norm=FOUR), -3), (dict(step_lr=FOUR), -3), (dict(grad_dtype=7), -1),
    (dict(state_bits=16), -1), (dict(drop=("p",)), -1), (dict(drop=("v",)), -1),
    (dict(state_bits=8, drop=("ms",)), -1), (dict(lens=(2 ** 43, 1)), -2),
])
def test_adamw_refusals(moe, kw, code):
    rc, _ = adamw_call(moe, **kw)
    assert rc == code and moe.lib.moe_last_error().decode() != ""


def test_adamw_nothing_to_do(moe):
    assert adamw_call(moe, n=0, lens=())[0] == 0
    assert adamw_call(moe, n=2, lens=(0, 0))[0] == 0


def test_adamw_check_finds_overlaps(moe):
    assert adamw_call(moe, check=True)[0] == 0
    assert adamw_call(moe, check=True, state_bits=8)[0] == 0
    # tensors 65536 bytes apart: 16384 fp32 elements fit, one more overlaps its neighbour
    assert adamw_call(moe, check=True, lens=(16384, 5))[0] == 0
    assert adamw_call(moe, check=True, lens=(16385, 5))[0] == -1
    assert "overlaps" in moe.lib.moe_last_error().decode()
    assert adamw_call(moe, check=True, lens=(16385, 0))[0] == 0


def test_binding_refuses_cpu_tensors(moe):
    import torch
    c = rcfg(moe, T=4, E=16)
    with pytest.raises(ValueError, match="CUDA"):
        moe.route(c, torch.zeros(4, 16))
    with pytest.raises(ValueError, match="CUDA"):
        moe.adamw_tensors(*[[torch.zeros(4)] for _ in range(4)])
    with pytest.raises(ValueError, match="entries"):
        moe.adamw_tensors([], [], [torch.zeros(4)], [])
    with pytest.raises(ValueError, match="bits"):
        moe.adamw_state([], bits=4)
    cfg = moe.make_config(4, 64, 64, 16, 8, 2)
    with pytest.raises(ValueError, match="shape"):
        moe.assign(cfg, torch.zeros(4, 7, dtype=torch.int32))
    with pytest.raises(TypeError, match="expert_idx"):
        moe.assign(cfg, torch.zeros(4, 8, dtype=torch.int64))


def test_expert_parallel_layer_refuses_more_choices_before_it_allocates(moe, monkeypatch):
    """The layer takes one or two choices: three are refused with that reason, not after (or by)
    the allocation of its buffers."""
    from sparse_mixture_experts_fwd_b200 import ep
    monkeypatch.setattr(ep.dist, "get_rank", lambda group=None: 0)
    monkeypatch.setattr(ep.dist, "get_world_size", lambda group=None: 2)

    def no_memory(*a, **k):
        raise AssertionError("allocated")

    monkeypatch.setattr(ep.torch, "empty", no_memory)
    with pytest.raises(moe.MoEError, match="k must be 1 or 2"):
        ep.ExpertParallelLayer(moe.make_config(64, 64, 64, 8, 3, 16), device="cpu")


WITHOUT_CUDA = """
import sys
sys.path.insert(0, ROOT)
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import sparse_mixture_experts_fwd_b200 as moe
class Stream:
    cuda_stream = 4096
asked = []
torch.cuda.current_stream = lambda device=None: (asked.append(device), Stream)[1]
torch.cuda.current_device = moe._current_device = lambda: 3
assert moe._stream() == 4096 and asked == [3]
assert moe.capacity(256, 8, 1.0) == 32
print("IMPORT_OK")
"""


def test_import_without_torchs_cuda_handles():
    """A torch without them (one built without CUDA) still imports the package, and the current
    stream then comes from torch's public functions."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", f"ROOT = {root!r}\n" + WITHOUT_CUDA],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "IMPORT_OK" in r.stdout, r.stdout + r.stderr
