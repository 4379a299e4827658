"""The binding's answers, on the host, to arguments of the latent attention's calls that are
missing, no tensors, or of the wrong number of axes: ValueError or TypeError with the argument's
name, before the library is called."""
import numpy as np
import pytest
import torch

from verify_spec_greedy_gb300 import _binding as b
from test_binding_checks import dev, lib  # noqa: F401
from test_latent_abi import append_args

BF, F16, I32 = torch.bfloat16, torch.float16, torch.int32
ATTN = dict(q=dev(2, 1, 3, 80, dtype=F16), cache=dev(5, 8, 80, dtype=F16),
            block_table=dev(2, 4, dtype=I32), kv_len=dev(2, dtype=I32), out=dev(2, 1, 3, 64, dtype=F16),
            scale=0.5, lse=dev(2, 1, 3), workspace=dev(512, dtype=torch.uint8))
PREFILL = dict(q=dev(6, 3, 80, dtype=BF), kv=dev(9, 3, 128, dtype=BF), rot=dev(9, 16, dtype=BF),
               cu_q=dev(3, dtype=I32), cu_k=dev(3, dtype=I32), out=dev(6, 3, 64, dtype=BF), scale=0.5)
CALLS = [("mtp_latent_append", append_args(),
          ["latent", "rot", "cos_sin", "tok_row", "positions", "block_table", "cache"]),
         ("mtp_latent_attn", ATTN, ["q", "cache", "block_table", "kv_len", "out"]),
         ("mtp_latent_prefill", PREFILL, ["q", "kv", "rot", "cu_q", "cu_k", "out"])]
REQUIRED = [(fn, args, name) for fn, args, names in CALLS for name in names]


@pytest.mark.parametrize("fn,args,name", REQUIRED, ids=[f"{f}-{n}" for f, _, n in REQUIRED])
def test_required_arguments(lib, fn, args, name):  # noqa: F811
    getattr(b, fn)(**args)
    assert len(lib.calls) == 1
    with pytest.raises(ValueError, match=rf"^{name} "):
        getattr(b, fn)(**{**args, name: None})
    for other in ([1, 2], np.zeros(tuple(args[name].shape), np.float32)):
        with pytest.raises(TypeError, match=rf"^{name} "):
            getattr(b, fn)(**{**args, name: other})
    assert len(lib.calls) == 1


@pytest.mark.parametrize("fn,args,name", [r for r in REQUIRED if r[2] not in
                                          ("tok_row", "positions", "kv_len", "cu_q", "cu_k")],
                         ids=lambda v: v if isinstance(v, str) else "")
def test_the_wrong_number_of_axes(lib, fn, args, name):  # noqa: F811
    t = args[name]
    for other in (t[None], dev(t.numel(), dtype=t.dtype) if t.dim() != 1 else t[None]):
        with pytest.raises(ValueError, match=rf"^{name} "):
            getattr(b, fn)(**{**args, name: other})
    assert lib.calls == []


@pytest.mark.parametrize("fn,name", [("mtp_latent_append", "norm_w"), ("mtp_latent_append", "q_rot"),
                                     ("mtp_latent_append", "q_out"), ("mtp_latent_attn", "lse"),
                                     ("mtp_latent_attn", "workspace"), ("mtp_latent_prefill", "lse")])
def test_optional_arguments_are_tensors(lib, fn, name):  # noqa: F811
    args = dict((f, a) for f, a, _ in CALLS)[fn]
    with pytest.raises(TypeError, match=rf"^{name} "):
        getattr(b, fn)(**{**args, name: [1.0]})
    assert lib.calls == []


def test_bounds_of_any_shape(lib):  # noqa: F811
    b.mtp_latent_prefill(**{**PREFILL, "cu_q": dev(1, 3, dtype=I32)})
    assert lib.calls[0][1][10] == 2
