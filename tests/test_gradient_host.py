"""The binding of the operators that make a node's gradient: devices, streams, workspaces and
shapes. Nothing here reaches a GPU."""
import pytest
import torch

from top_gradient_compression_gb300 import api

from test_training_host import calls, placed  # noqa: F401 (a fixture)

HALF = torch.bfloat16
I32 = torch.int32


def stored(*shape):
    *lead, dim = shape
    return api.Checkpoint8(placed(*lead, (dim + 15) // 16 * 16, dtype=torch.int8),
                           placed(*lead, (dim + 127) // 128, dtype=torch.uint8), dim, HALF)


def space():
    return placed(4096, dtype=torch.uint8)


def h(*shape):
    return placed(*shape, dtype=HALF)


def operands(name):
    """(function, operands as keywords, entry point)."""
    heads = {"q": h(5, 4, 16), "k": h(5, 2, 16), "positions": placed(5, dtype=I32),
             "freqs": placed(8), "q_weight": h(16), "k_weight": h(16), "q_out": h(5, 4, 16),
             "k_out": h(5, 2, 16)}
    experts = {"weight": h(3, 8, 16), "offsets": placed(4, dtype=I32), "ws": space()}
    back = {"dy": h(6, 8), "dx": h(6, 16), "dweight": placed(3, 8, 16), **experts}
    turned = {k: v for k, v in heads.items() if not k.endswith("_out")}
    return {
        "checkpoint8": (api.checkpoint8, {"x": h(4, 24), "out": stored(4, 24)},
                        "sparcml_checkpoint8"),
        "restore8": (api.restore8, {"x": stored(4, 24), "out": h(4, 24)}, "sparcml_restore8"),
        "norm": (api.layer_norm_backward,
                 {"dy": h(4, 24), "x": stored(4, 24), "mean": placed(4), "rstd": placed(4),
                  "weight": h(24), "dx": h(4, 24), "dweight": placed(24), "dbias": placed(24),
                  "ws": space()}, "sparcml_layer_norm_backward8"),
        "experts": (api.expert_linear, {"x": h(6, 16), "out": h(6, 8), **experts},
                    "sparcml_expert_linear"),
        "experts back": (api.expert_linear_backward, {"x": h(6, 16), **back},
                         "sparcml_expert_linear_backward"),
        "experts back 8": (api.expert_linear_backward, {"x": stored(6, 16), **back},
                           "sparcml_expert_linear_backward8"),
        "heads": (api.head_norm_rotary, heads, "sparcml_head_norm_rotary"),
        "heads back": (api.head_norm_rotary_backward,
                       {"dq": h(5, 4, 16), "dk": h(5, 2, 16), **turned, "dq_out": h(5, 4, 16),
                        "dk_out": h(5, 2, 16), "dq_weight": placed(16), "dk_weight": placed(16),
                        "ws": space()}, "sparcml_head_norm_rotary_backward"),
    }[name]


NAMES = ["checkpoint8", "restore8", "norm", "experts", "experts back", "experts back 8", "heads",
         "heads back"]


def tensors(v):
    return [v.codes, v.exponents] if isinstance(v, api.Checkpoint8) else [v]


@pytest.mark.parametrize("name", NAMES)
def test_operands_on_two_devices_are_refused(name, calls):  # noqa: F811
    for odd in operands(name)[1]:
        for part in range(len(tensors(operands(name)[1][odd]))):
            f, args, _ = operands(name)
            tensors(args[odd])[part].index = 1
            with pytest.raises(ValueError, match="one device"):
                f(**args)
    assert calls == []


@pytest.mark.parametrize("name", NAMES)
def test_the_operands_device_is_current_during_the_call(name, calls):  # noqa: F811
    for index in (0, 1):
        f, args, entry = operands(name)
        for v in args.values():
            for t in tensors(v):
                t.index = index
        f(**args)
    assert calls == [(entry, i, 1000 + i) for i in (0, 1)]


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_device_is_refused(name, calls):  # noqa: F811
    class Stream:
        device = torch.device("cuda", 1)
    f, args, _ = operands(name)
    with pytest.raises(ValueError, match="stream"):
        f(**args, stream=Stream())
    assert calls == []


@pytest.mark.parametrize("name", [n for n in NAMES if "8" not in n or "back" in n if n != "heads"])
def test_a_workspace_has_to_be_contiguous_device_memory(name, calls):  # noqa: F811
    f, args, _ = operands(name)
    args["ws"] = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(TypeError, match="ws"):
        f(**args)
    args["ws"] = placed(1, dtype=torch.uint8).expand(4096)  # one byte
    with pytest.raises(ValueError, match="ws"):
        f(**args)
    assert calls == []


REFUSED = [
    ("checkpoint8", {"x": torch.zeros(4, 24, dtype=HALF)}),      # on the host
    ("checkpoint8", {"x": placed(4, 24, dtype=torch.float64)}),
    ("checkpoint8", {"x": h(4, 48)[:, ::2]}),                    # not contiguous
    ("checkpoint8", {"out": stored(4, 25)}),
    ("checkpoint8", {"x": placed(4, 24)}),                       # fp32, and out of bf16
    ("restore8", {"out": h(4, 25)}),
    ("restore8", {"x": api.Checkpoint8(placed(4, 24, dtype=torch.int8),
                                       placed(4, 1, dtype=torch.uint8), 24, HALF)}),
    ("restore8", {"x": api.Checkpoint8(placed(4, 32, dtype=torch.int8),
                                       placed(4, 2, dtype=torch.uint8), 24, HALF)}),
    ("restore8", {"x": api.Checkpoint8(placed(4, 32, dtype=torch.uint8),
                                       placed(4, 1, dtype=torch.uint8), 24, HALF)}),
    ("restore8", {"x": api.Checkpoint8(placed(4, 32, dtype=torch.int8),
                                       placed(4, 1, dtype=torch.uint8), 24, torch.int8)}),
    ("norm", {"dy": h(4, 25)}), ("norm", {"dy": placed(4, 24)}), ("norm", {"mean": placed(5)}),
    ("norm", {"dweight": placed(23)}), ("norm", {"weight": h(25)}), ("norm", {"dx": h(5, 24)}),
    ("experts", {"x": placed(6, 16)}),                           # fp32
    ("experts", {"x": h(6, 17)}), ("experts", {"x": h(2, 6, 16)}),
    ("experts", {"weight": placed(3, 8, 16, dtype=torch.float16)}),
    ("experts", {"weight": h(8, 16)}),                           # one matrix, offsets of three
    ("experts", {"weight": h(3, 8, 32)[..., ::2]}),
    ("experts", {"offsets": None}), ("experts", {"offsets": placed(3, dtype=I32)}),
    ("experts", {"offsets": placed(4, dtype=torch.int64)}), ("experts", {"out": h(6, 9)}),
    ("experts", {"out": placed(6, 8)}),
    ("experts back", {"dy": h(6, 9)}), ("experts back", {"x": h(5, 16)}),
    ("experts back", {"dx": h(6, 15)}), ("experts back", {"dweight": h(3, 8, 16)}),
    ("experts back", {"dweight": placed(8, 16)}),
    ("experts back", {"dweight": None, "accumulate": True}),
    ("experts back 8", {"x": stored(6, 17)}), ("experts back 8", {"x": stored(7, 16)}),
    ("experts back 8", {"dy": placed(6, 8, dtype=torch.float16)}),
    ("heads", {"q": h(5, 64)}), ("heads", {"k": h(4, 2, 16)}), ("heads", {"k": h(5, 2, 18)}),
    ("heads", {"k": placed(5, 2, 16)}), ("heads", {"q": None, "k": None}),
    ("heads", {"positions": placed(5)}), ("heads", {"positions": placed(4, dtype=I32)}),
    ("heads", {"positions": placed(10, dtype=I32)[::2]}), ("heads", {"freqs": placed(9)}),
    ("heads", {"freqs": placed(8, dtype=torch.float64)}), ("heads", {"q_weight": h(15)}),
    ("heads", {"q_weight": placed(16)}), ("heads", {"q_out": h(5, 4, 17)}),
    ("heads", {"q": h(5, 4, 32)[..., ::2]}),
    ("heads back", {"dq": None}), ("heads back", {"k": None}), ("heads back", {"dq": h(5, 5, 16)}),
    ("heads back", {"dq_weight": placed(15)}), ("heads back", {"dq_weight": h(16)}),
    ("heads back", {"dk_weight": None, "accumulate": True}),
]


@pytest.mark.parametrize("name,change", REFUSED)
def test_refusals(name, change, calls):  # noqa: F811
    f, args, _ = operands(name)
    args.update(change)
    with pytest.raises((TypeError, ValueError)):
        f(**args)
    assert calls == []


def test_outputs_are_made_where_none_are_given(calls, monkeypatch):  # noqa: F811
    monkeypatch.setattr(torch, "empty", lambda *shape, dtype, device: placed(*shape, dtype=dtype))
    x = h(2, 3, 24)
    c = api.checkpoint8(x)
    assert c.codes.shape == (2, 3, 32) and c.exponents.shape == (2, 3, 1) and c.dtype == HALF
    assert c.shape == (2, 3, 24) and "2, 3, 24" in repr(c)
    assert api.restore8(c).dtype == HALF and api.restore8(c, dtype=torch.float32).shape == x.shape
    _, args, _ = operands("experts")
    del args["out"]
    y = api.expert_linear(**args)
    assert y.shape == (6, 8) and y.dtype == HALF
    _, args, _ = operands("experts back 8")
    del args["dx"], args["dweight"]
    dx, dw = api.expert_linear_backward(**args)
    assert dx.shape == (6, 16) and dw.shape == (3, 8, 16) and dw.dtype == torch.float32
    assert api.expert_linear_backward(**args, need_dx=False)[0] is None
    assert api.expert_linear_backward(**args, need_dweight=False)[1] is None
    _, args, _ = operands("heads")
    q, k = api.head_norm_rotary(**{**args, "q_out": None, "k": None, "k_out": None})
    assert q.shape == (5, 4, 16) and k is None
